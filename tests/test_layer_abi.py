"""The C ABI of the norm, the 8-bit cache and attention (include/lora_layer.h):
every declared entry point is exported and bound, what the host can see to be
wrong is refused with the documented status before anything is launched, the
sizes of plans and workspaces are right, and the binding passes on only what
fits.  CPU only."""
import ctypes
import math
import os
import re

import pytest
import torch

import rank_sgmv_bgmv_amd as L
from test_base_abi import BF16, EINVAL, ESHAPE, EUNSUPPORTED, EWORKSPACE, F32, FAKE, MANY, ROOT, Stand, launched, lib  # noqa: F401


def test_declared_entry_points_are_exported_and_bound(lib):  # noqa: F811
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lora_layer.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(lora_[a-z_]+)\s*\(", text))
    assert len(names) == 8, names
    for name in names:
        assert hasattr(lib, name) and callable(getattr(L, name)), name


def test_structures_are_those_of_the_header(lib):  # noqa: F811
    """Sizes as the C compiler lays them out on this platform: members in order, none missing."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lora_layer.h")).read(), flags=re.S)
    found = re.findall(r"typedef struct \{(.*?)\}\s*(lora_\w+);", text, flags=re.S)
    assert {n for _, n in found} == {"lora_norm", "lora_cache", "lora_heads", "lora_attention", "lora_attention_batch"}
    sizes = {"int32_t": 4, "int64_t": 8, "float": 4, "double": 8, "lora_dtype": 4}
    for body, name in found:
        members = []
        for line in body.split(";"):
            m = re.match(r"\s*(?:const\s+)?(\w+)\s+(.*)$", line.strip(), flags=re.S)
            if m:
                members += [(v.strip(" *"), 8 if "*" in v else sizes[m.group(1)]) for v in m.group(2).split(",")]
        kind = getattr(L, name)
        assert [(f, ctypes.sizeof(t)) for f, t in kind._fields_] == members, name


def norm(lib, n=None, **kw):  # noqa: F811
    nn = dict(weight=FAKE * 9000, eps=1e-5, d=64)
    nn.update(n or {})
    nn = L.lora_norm(*nn.values())
    v = dict(x=FAKE, ldx=64, r=FAKE * 2, ldr=64, total=FAKE * 3, ldt=64, y=FAKE * 4, ldy=64, q=FAKE * 5, ldq=64,
             scale=FAKE * 6, rows=8, dtype=BF16, stream=None)
    v.update(kw)
    return lib.lora_norm_apply(ctypes.addressof(nn), *v.values())


@pytest.mark.parametrize("n, kw, status", [
    ({}, dict(rows=0, x=None, y=None), 0),
    ({}, dict(dtype=5), EINVAL), ({"weight": None}, {}, EINVAL), ({"weight": FAKE + 2}, {}, EINVAL),
    ({"eps": -1.0}, {}, EINVAL), ({"eps": math.nan}, {}, EINVAL), ({"eps": math.inf}, {}, EINVAL),
    ({"d": 0}, {}, ESHAPE), ({"d": 65537}, {}, EUNSUPPORTED),
    ({}, dict(rows=-1), ESHAPE), ({}, dict(x=None), EINVAL), ({}, dict(y=None, q=None, scale=None), EINVAL),
    ({}, dict(q=None), EINVAL), ({}, dict(scale=None), EINVAL), ({}, dict(r=None), EINVAL),
    ({}, dict(ldx=63), ESHAPE), ({}, dict(ldr=63), ESHAPE), ({}, dict(ldt=63), ESHAPE), ({}, dict(ldy=63), ESHAPE),
    ({}, dict(ldq=63), ESHAPE), ({}, dict(ldy=1 << 60), ESHAPE),
    ({}, dict(x=FAKE + 1), EINVAL), ({}, dict(y=FAKE * 4 + 1), EINVAL), ({}, dict(scale=FAKE * 6 + 1), EINVAL),
    ({}, dict(dtype=F32, r=FAKE * 2 + 2), EINVAL),
    # overlap of what is written
    ({}, dict(y=FAKE + 2), EINVAL), ({}, dict(total=FAKE + 2), EINVAL), ({}, dict(y=FAKE * 2), EINVAL),
    ({}, dict(y=FAKE * 3), EINVAL), ({}, dict(q=FAKE), EINVAL), ({}, dict(q=FAKE * 4 + 1000), EINVAL),
    ({}, dict(scale=FAKE * 5 + 8), EINVAL), ({}, dict(y=FAKE * 9000), EINVAL), ({}, dict(scale=FAKE * 9000), EINVAL),
    # in place, but at another stride
    ({}, dict(y=FAKE, ldy=72), EINVAL), ({}, dict(total=FAKE * 2, ldt=72), EINVAL),
    # the total over x, and y over both
    ({}, dict(total=FAKE, y=FAKE), EINVAL),
])
def test_norm_refusals(lib, n, kw, status):  # noqa: F811
    assert norm(lib, n, **kw) == status


def test_norm_without_norm(lib):  # noqa: F811
    assert lib.lora_norm_apply(None, FAKE, 64, None, 0, None, 0, FAKE * 2, 64, None, 0, None, 8, BF16, None) == EINVAL


def test_pitch(lib):  # noqa: F811
    assert [lib.lora_cache_pitch(d) for d in (-1, 0, 1, 16, 17, 80, 128, 256, 257)] == [0, 0, 16, 16, 32, 80, 128, 256, 0]


PAGE = 2 * 16 * 64  # bytes of a page of the cache below: 2 heads, 16 slots, rows of 64


def cache(**kw):
    v = dict(k=FAKE * 1000, v=FAKE * 2000, k_scale=FAKE * 3000, v_scale=FAKE * 4000, k_page=PAGE, v_page=PAGE, k_scale_page=32,
             v_scale_page=32, n_pages=10, n_heads=2, page_size=16, head_dim=64)
    v.update(kw)
    return L.lora_cache(*v.values())


def heads(data, token=128, head=64):
    return L.lora_heads(data, token, head)


def call_cache(lib, write, c=None, k_heads=None, v_heads=None, **kw):  # noqa: F811
    c = cache() if c is None else c
    k = heads(FAKE * 10) if k_heads is None else k_heads
    v = heads(FAKE * 20) if v_heads is None else v_heads
    a = dict(slots=FAKE, T=8, k=ctypes.addressof(k), v=ctypes.addressof(v), dtype=BF16, stream=None)
    a.update(kw)
    f = lib.lora_cache_write if write else lib.lora_cache_read
    return f(ctypes.addressof(c), *a.values())


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("c, k, kw, status", [
    ({}, {}, dict(T=0, slots=None, k=None, v=None), 0),
    ({}, {}, dict(dtype=9), EINVAL), ({}, {}, dict(T=-1), ESHAPE), ({}, {}, dict(slots=None), EINVAL),
    ({}, {}, dict(slots=FAKE + 2), EINVAL), ({}, {}, dict(k=None), EINVAL), ({}, {}, dict(v=None), EINVAL),
    ({"k": None}, {}, {}, EINVAL), ({"v": None}, {}, {}, EINVAL), ({"k_scale": None}, {}, {}, EINVAL),
    ({"v_scale": None}, {}, {}, EINVAL), ({"k": FAKE * 1000 + 8}, {}, {}, EINVAL), ({"v_scale": FAKE * 4000 + 4}, {}, {}, EINVAL),
    ({"k_page": PAGE - 16}, {}, {}, ESHAPE), ({"v_page": PAGE + 8}, {}, {}, EINVAL), ({"k_scale_page": 34}, {}, {}, EINVAL),
    ({"v_scale_page": 31}, {}, {}, ESHAPE), ({"k_page": -PAGE}, {}, {}, ESHAPE), ({"k_page": 1 << 62}, {}, {}, ESHAPE),
    ({"n_pages": 0}, {}, {}, ESHAPE), ({"n_heads": 0}, {}, {}, ESHAPE), ({"head_dim": 0}, {}, {}, ESHAPE),
    ({"head_dim": 257}, {}, {}, EUNSUPPORTED), ({"n_heads": 65536}, {}, {}, EUNSUPPORTED),
    ({"page_size": 8}, {}, {}, ESHAPE), ({"page_size": 24}, {}, {}, ESHAPE), ({"page_size": 2048}, {}, {}, ESHAPE),
    ({}, {"data": None}, {}, EINVAL), ({}, {"data": FAKE * 10 + 1}, {}, EINVAL), ({}, {"token": -1}, {}, ESHAPE),
    ({}, {"head": 1 << 60}, {}, ESHAPE), ({}, {"data": FAKE * 1000 + 64}, {}, EINVAL), ({}, {"data": FAKE * 3000}, {}, EINVAL),
])
def test_cache_refusals(lib, write, c, k, kw, status):  # noqa: F811
    k = L.lora_heads(*{**dict(data=FAKE * 10, token=128, head=64), **k}.values())
    assert call_cache(lib, write, cache(**c), k, **kw) == status


def test_cache_write_refusals(lib):  # noqa: F811
    """Arrays of the cache that meet, and slots in it."""
    assert call_cache(lib, True, cache(v=FAKE * 1000 + 1024)) == EINVAL
    assert call_cache(lib, True, cache(v_scale=FAKE * 1000 + 64)) == EINVAL
    assert call_cache(lib, True, slots=FAKE * 2000) == EINVAL
    # pages side by side, the second array's first page 16 bytes early
    wide = dict(k_page=2 * PAGE, v_page=2 * PAGE)
    assert call_cache(lib, True, cache(v=FAKE * 1000 + PAGE - 16, **wide)) == EINVAL


def test_cache_read_refusals(lib):  # noqa: F811
    """Values of the outputs that share a place, and outputs that meet each other or the slots."""
    assert call_cache(lib, False, k_heads=heads(FAKE * 10, token=64)) == ESHAPE
    assert call_cache(lib, False, v_heads=heads(FAKE * 10 + 64)) == EINVAL
    assert call_cache(lib, False, v_heads=heads(FAKE)) == EINVAL


def attend(lib, att=None, c=None, b=None, q_heads=None, out_heads=None, f=None, **kw):  # noqa: F811
    att = L.lora_attention(*{**dict(n_heads=4, window=0, sinks=0, scale=0.125, dtype=BF16), **(att or {})}.values())
    c = cache(**(c or {}))
    b = L.lora_attention_batch(*{**dict(n_tokens=8, n_seqs=3, max_q=4, max_pages=6, q_off=FAKE * 50, lens=FAKE * 51,
                                        pages=FAKE * 52, ld_pages=6, tree=None), **(b or {})}.values())
    refs = [ctypes.addressof(v) for v in (att, c, b)]
    if f is not None:
        return f(*refs)
    q = heads(FAKE * 10, 256) if q_heads is None else q_heads
    out = heads(FAKE * 20, 256) if out_heads is None else out_heads
    v = dict(plan=FAKE * 100, plan_bytes=1 << 20, q=ctypes.addressof(q), out=ctypes.addressof(out), ws=FAKE * 200,
             ws_bytes=1 << 30, stream=None)
    v.update(kw)
    return lib.lora_attention_apply(*refs, *v.values())


SIZES = [
    ({"n_heads": 0}, {}, {}, ESHAPE), ({"n_heads": 3}, {}, {}, ESHAPE), ({"n_heads": 65536}, {"n_heads": 1}, {}, EUNSUPPORTED),
    ({"window": -1}, {}, {}, ESHAPE), ({"sinks": -1}, {}, {}, ESHAPE), ({"dtype": 4}, {}, {}, EINVAL),
    ({"scale": 0.0}, {}, {}, ESHAPE), ({"scale": -1.0}, {}, {}, ESHAPE), ({"scale": math.nan}, {}, {}, ESHAPE),
    ({"scale": math.inf}, {}, {}, ESHAPE),
    ({}, {"page_size": 20}, {}, ESHAPE), ({}, {"head_dim": 300}, {}, EUNSUPPORTED), ({}, {"n_pages": 0}, {}, ESHAPE),
    ({}, {}, {"n_tokens": -1}, ESHAPE), ({}, {}, {"n_seqs": -1}, ESHAPE), ({}, {}, {"max_q": 0}, ESHAPE),
    ({}, {}, {"max_pages": 0}, ESHAPE), ({}, {}, {"ld_pages": 5}, ESHAPE), ({}, {}, {"ld_pages": 1 << 60}, ESHAPE),
    ({}, {}, {"max_pages": (1 << 26) + 1, "ld_pages": 1 << 30}, EUNSUPPORTED),
    ({}, {}, {"tree": FAKE * 53, "max_q": 65}, EUNSUPPORTED),
    ({}, {}, {"n_tokens": 1 << 29}, EUNSUPPORTED), ({}, {}, {"n_seqs": (1 << 24) + 1}, EUNSUPPORTED),
]


@pytest.mark.parametrize("att, c, b, status", SIZES)
def test_attention_sizes(lib, att, c, b, status):  # noqa: F811
    assert attend(lib, att, c, b) == status
    assert attend(lib, att, c, b, f=lib.lora_attention_plan_size) == 0
    assert attend(lib, att, c, b, f=lib.lora_attention_workspace_size) == 0
    assert attend(lib, att, c, b, f=lambda *r: lib.lora_attention_plan(*r, FAKE * 100, 1 << 30, None)) == status


@pytest.mark.parametrize("c, b, kw, status", [
    ({}, {"n_tokens": 0}, dict(plan=None, ws=None, q=None, out=None), 0),
    ({}, {"n_seqs": 0}, dict(plan=None, ws=None), 0),
    ({}, {}, dict(plan=None), EWORKSPACE), ({}, {}, dict(plan_bytes=100), EWORKSPACE), ({}, {}, dict(ws=None), EWORKSPACE),
    ({}, {}, dict(plan=FAKE * 100 + 8), EINVAL), ({}, {}, dict(ws=FAKE * 200 + 8), EINVAL),
    ({}, {}, dict(q=None), EINVAL), ({}, {}, dict(out=None), EINVAL),
    ({"k": None}, {}, {}, EINVAL), ({"v_scale_page": 16}, {}, {}, ESHAPE),
    ({}, {"pages": None}, {}, EINVAL), ({}, {"pages": FAKE + 2}, {}, EINVAL), ({}, {"tree": FAKE + 4}, {}, EINVAL),
    # out over the cache, the pages, the plan, the workspace
    ({}, {"pages": FAKE * 20}, {}, EINVAL), ({}, {"tree": FAKE * 20}, {}, EINVAL), ({"k": FAKE * 20}, {}, {}, EINVAL),
    ({}, {}, dict(plan=FAKE * 20), EINVAL), ({}, {}, dict(ws=FAKE * 20), EINVAL), ({}, {}, dict(ws=FAKE * 10), EINVAL),
    ({}, {}, dict(ws=FAKE * 100), EINVAL), ({}, {}, dict(ws=FAKE * 52), EINVAL), ({}, {}, dict(ws=FAKE * 2000), EINVAL),
])
def test_attention_refusals(lib, c, b, kw, status):  # noqa: F811
    assert attend(lib, None, c, b, **{**dict(ws_bytes=4096), **kw}) == status


def test_attention_needs_its_workspace(lib):  # noqa: F811
    """Where long sequences may be cut their parts need room."""
    b = {"max_pages": 1000, "ld_pages": 1000}
    need = attend(lib, None, {}, b, f=lib.lora_attention_workspace_size)
    assert need > 1 << 16
    assert attend(lib, None, {}, b, ws_bytes=1 << 16) == EWORKSPACE


@pytest.mark.parametrize("q, out, status", [
    (heads(FAKE * 10 + 1, 256), None, EINVAL), (heads(FAKE * 10, -256), None, ESHAPE), (None, heads(FAKE * 20, 128), ESHAPE),
    (None, heads(FAKE * 20, 256, 0), ESHAPE), (None, heads(FAKE * 10 + 128, 256), EINVAL),
    (None, heads(FAKE * 10, 512), ESHAPE), (None, heads(None, 256), EINVAL),
])
def test_attention_heads_refusals(lib, q, out, status):  # noqa: F811
    assert attend(lib, q_heads=q, out_heads=out) == status


@pytest.mark.parametrize("b, plan, n, status", [
    ({"q_off": None}, FAKE * 100, 1 << 20, EINVAL), ({"lens": None}, FAKE * 100, 1 << 20, EINVAL),
    ({"lens": FAKE + 1}, FAKE * 100, 1 << 20, EINVAL), ({}, None, 1 << 20, EWORKSPACE), ({}, FAKE * 100, 256, EWORKSPACE),
    ({}, FAKE * 100 + 4, 1 << 20, EINVAL), ({}, FAKE * 50, 1 << 16, EINVAL), ({}, FAKE * 51, 1 << 16, EINVAL),
])
def test_plan_refusals(lib, b, plan, n, status):  # noqa: F811
    assert attend(lib, b=b, f=lambda *r: lib.lora_attention_plan(*r, plan, n, None)) == status


def test_sizes_grow_with_the_batch(lib):  # noqa: F811
    size = lambda **b: (attend(lib, b=b, f=lib.lora_attention_plan_size), attend(lib, b=b, f=lib.lora_attention_workspace_size))  # noqa: E731
    few, more, long = size(), size(n_tokens=800, n_seqs=300), size(max_pages=4096, ld_pages=4096)
    assert 0 < few[0] < more[0] and few[1] <= long[1] and few[0] <= long[0]
    # nothing is cut, so there is nothing to keep
    assert few[1] == 256


def stand_cache(n_pages=4, heads=2, page=16, d=64):
    pitch = L.lora_cache_pitch(d)
    k, v = (Stand(torch.int8, n_pages, heads, page, pitch) for _ in range(2))
    ks, vs = (Stand(torch.float32, n_pages, heads, page) for _ in range(2))
    return L.Cache(k, v, ks, vs, d)


def stand_batch(T=8, S=3, tree=None, pages=None):
    i = torch.int32
    return L.AttentionBatch(T, Stand(i, S + 1), Stand(i, S), Stand(i, S, 6) if pages is None else pages, 4, tree)


def bf(*shape, **kw):
    return Stand(torch.bfloat16, *shape, **kw)


def test_what_the_binding_passes(launched):  # noqa: F811
    c, b = stand_cache(), stand_batch()
    att = L.Attention(4, 0.125, window=100, sinks=4)
    plan, ws = Stand(torch.uint8, 1 << 16), Stand(torch.uint8, 1 << 16)
    L.lora_attention_plan(att, c, b, plan)
    assert launched[-1] == (att.ref, c.ref, b.ref, FAKE, 1 << 16)
    L.lora_attention_apply(att, c, b, plan, bf(8, 4, 64), bf(8, 4, 64, strides=(64, 512, 1)), ws)
    *head, qb, ob, wp, wn = launched[-1]
    assert L.lora_heads.from_buffer_copy(qb).token == 256 and L.lora_heads.from_buffer_copy(ob).head == 512 and wn == 1 << 16
    L.lora_cache_write(c, Stand(torch.int32, 8), bf(8, 2, 64), bf(8, 2, 64))
    assert launched[-1][0] == c.ref and launched[-1][2] == 8 and launched[-1][5] == BF16
    n = L.Norm(Stand(torch.float32, 64), 1e-6)
    L.lora_norm_apply(n, bf(1, 64, strides=(1, 1)), y=bf(1, 64))
    assert launched[-1][1:5] == (FAKE, 64, None, 0) and launched[-1][7:9] == (FAKE, 64)


@pytest.mark.parametrize("call", [
    lambda c, b: L.Norm(torch.ones(4), 1e-5),
    lambda c, b: L.Norm(Stand(torch.bfloat16, 64), 1e-5),
    lambda c, b: L.lora_norm_apply(L.Norm(Stand(torch.float32, 64), 0.0), bf(8, 63), y=bf(8, 63)),
    lambda c, b: L.lora_norm_apply(L.Norm(Stand(torch.float32, 64), 0.0), bf(8, 64), y=bf(7, 64)),
    lambda c, b: L.lora_norm_apply(L.Norm(Stand(torch.float32, 64), 0.0), bf(8, 64), y=Stand(torch.float32, 8, 64)),
    lambda c, b: L.lora_norm_apply(L.Norm(Stand(torch.float32, 64), 0.0), bf(8, 64), y=bf(8, 64), residual=bf(8, 128)),
    lambda c, b: L.lora_norm_apply(L.Norm(Stand(torch.float32, 64), 0.0), bf(8, 64), q=Stand(torch.uint8, 8, 64), scale=Stand(torch.float32, 8)),
    lambda c, b: L.lora_norm_apply(L.Norm(Stand(torch.float32, 64), 0.0), bf(8, 64), q=Stand(torch.int8, 8, 64), scale=Stand(torch.float32, 7)),
    lambda c, b: L.lora_norm_apply(L.Norm(Stand(torch.float32, 64), 0.0), Stand(torch.float16, 8, 64), y=Stand(torch.float16, 8, 64)),
    lambda c, b: L.lora_norm_apply(L.Norm(Stand(torch.float32, 64), 0.0), bf(MANY, 64), y=bf(MANY, 64)),
    lambda c, b: L.Cache(*[torch.zeros(1)] * 4, 64),
    lambda c, b: L.Cache(Stand(torch.int8, 4, 2, 16, 64), Stand(torch.int8, 4, 2, 16, 64), Stand(torch.float32, 4, 2, 16), Stand(torch.float32, 4, 2, 16), 80),
    lambda c, b: L.Cache(Stand(torch.int8, 4, 2, 16, 64), Stand(torch.int8, 4, 2, 16, 64, strides=(4096, 64, 128, 1)), Stand(torch.float32, 4, 2, 16), Stand(torch.float32, 4, 2, 16), 64),
    lambda c, b: L.Cache(Stand(torch.int8, 4, 2, 16, 64), Stand(torch.int8, 3, 2, 16, 64), Stand(torch.float32, 4, 2, 16), Stand(torch.float32, 4, 2, 16), 64),
    lambda c, b: L.Cache(Stand(torch.int8, 4, 2, 16, 64), Stand(torch.int8, 4, 2, 16, 64), Stand(torch.float64, 4, 2, 16), Stand(torch.float32, 4, 2, 16), 64),
    lambda c, b: L.Cache(Stand(torch.int8, MANY, 2, 16, 64), Stand(torch.int8, MANY, 2, 16, 64), Stand(torch.float32, MANY, 2, 16), Stand(torch.float32, MANY, 2, 16), 64),
    lambda c, b: L.lora_cache_write(c, Stand(torch.int64, 8), bf(8, 2, 64), bf(8, 2, 64)),
    lambda c, b: L.lora_cache_write(c, Stand(torch.int32, 8), bf(7, 2, 64), bf(8, 2, 64)),
    lambda c, b: L.lora_cache_write(c, Stand(torch.int32, 8), bf(8, 2, 64), Stand(torch.float32, 8, 2, 64)),
    lambda c, b: L.lora_cache_read(c, Stand(torch.int32, 8), bf(8, 2, 64, strides=(128, 1, 2)), bf(8, 2, 64)),
    lambda c, b: L.lora_cache_read(c, Stand(torch.int32, MANY), bf(MANY, 2, 64), bf(MANY, 2, 64)),
    lambda c, b: L.lora_cache_pitch(MANY),
    lambda c, b: L.Attention(4, 1.0, dtype=torch.float16),
    lambda c, b: L.Attention(MANY, 1.0), lambda c, b: L.Attention(4, 1.0, window=MANY), lambda c, b: L.Attention(4, 1.0, sinks=MANY),
    lambda c, b: stand_batch(T=MANY), lambda c, b: stand_batch(pages=Stand(torch.int64, 3, 6)),
    lambda c, b: stand_batch(pages=Stand(torch.int32, 3, 6, strides=(1, 3))), lambda c, b: stand_batch(pages=torch.zeros(3, 6, dtype=torch.int32)),
    lambda c, b: stand_batch(tree=Stand(torch.int64, 7)), lambda c, b: stand_batch(tree=Stand(torch.int32, 8)),
    lambda c, b: L.AttentionBatch(8, Stand(torch.int32, 3), Stand(torch.int32, 3), Stand(torch.int32, 3, 6), 4),
    lambda c, b: L.AttentionBatch(8, Stand(torch.int32, 4), Stand(torch.int32, 2), Stand(torch.int32, 3, 6), 4),
    lambda c, b: L.lora_attention_apply(L.Attention(4, 1.0), c, b, Stand(torch.uint8, 9999), bf(8, 4, 64), bf(8, 4, 32), Stand(torch.uint8, 9999)),
    lambda c, b: L.lora_attention_apply(L.Attention(4, 1.0), c, b, Stand(torch.int8, 9999), bf(8, 4, 64), bf(8, 4, 64), Stand(torch.uint8, 9999)),
    lambda c, b: L.lora_attention_apply(L.Attention(4, 1.0), c, b, Stand(torch.uint8, 9999), bf(7, 4, 64), bf(8, 4, 64), Stand(torch.uint8, 9999)),
    lambda c, b: L.lora_attention_apply(L.Attention(2, 1.0), c, b, Stand(torch.uint8, 9999), bf(8, 4, 64), bf(8, 4, 64), Stand(torch.uint8, 9999)),
    lambda c, b: L.lora_attention_plan_size(L.Attention(3, 1.0), c, b), lambda c, b: L.new_attention_workspace(L.Attention(4, -1.0), c, b),
])
def test_what_the_binding_refuses(launched, call):  # noqa: F811
    c, b = stand_cache(), stand_batch()
    with pytest.raises(L.LoraError):
        call(c, b)
    assert not launched
