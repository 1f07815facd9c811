"""The C ABI around a LoRA layer (include/lora_base.h): every declared entry
point is exported and bound, what the host can see to be wrong is refused with
the documented status before anything is launched, and the host-side results
(workspace sizes, rotary frequencies) are right.  CPU only."""
import ctypes
import math
import os
import re
import sys

import numpy as np
import pytest
import torch

import rank_sgmv_bgmv_amd as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, ESHAPE, EWORKSPACE, EUNSUPPORTED = -1, -2, -3, -4
FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced
BF16, F32 = L.LORA_BF16, L.LORA_F32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from rank_sgmv_bgmv_amd import build
        build.build()
    return L.lib()


def test_declared_entry_points_are_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lora_base.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(lora_[a-z_]+)\s*\(", text))
    assert len(names) == 6, names
    for name in names:
        assert hasattr(lib, name) and hasattr(L, name), name


def weight(**kw):
    v = dict(W=FAKE * 100, scale=FAKE * 8000, bias=None, ldw=64, d_in=64, d_out=32)
    v.update(kw)
    return L.lora_base_weight(*v.values())


def quantize(lib, **kw):
    v = dict(x=FAKE, ldx=64, dtype=BF16, rows=8, d=64, q=FAKE * 10, ldq=64, scale=FAKE * 20, stream=None)
    v.update(kw)
    return lib.lora_quantize_rows(*v.values())


@pytest.mark.parametrize("kw, status", [
    (dict(rows=0, x=None, q=None, scale=None), 0),
    (dict(dtype=7), EINVAL), (dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(rows=-1), ESHAPE), (dict(d=0), ESHAPE), (dict(ldx=63), ESHAPE), (dict(ldq=63), ESHAPE),
    (dict(ldx=-64), ESHAPE), (dict(ldx=1 << 62), ESHAPE),
    (dict(x=FAKE + 1), EINVAL), (dict(dtype=F32, x=FAKE + 2), EINVAL), (dict(scale=FAKE * 20 + 2), EINVAL),
    (dict(q=FAKE + 1023), EINVAL), (dict(scale=FAKE + 1020), EINVAL), (dict(scale=FAKE * 10 + 508), EINVAL),
])
def test_quantize_refusals(lib, kw, status):
    assert quantize(lib, **kw) == status


def product(lib, w=None, **kw):
    v = dict(q=FAKE, ldq=64, q_scale=FAKE * 2, T=8, y=FAKE * 3, ldy=32, dtype=BF16, stream=None)
    v.update(kw)
    w = weight() if w is None else w
    return lib.lora_base_product(ctypes.addressof(w), *v.values())


@pytest.mark.parametrize("w, kw, status", [
    ({}, dict(T=0, q=None, q_scale=None, y=None), 0),
    ({}, dict(dtype=2), EINVAL), ({}, dict(q=None), EINVAL), ({}, dict(q_scale=None), EINVAL), ({}, dict(y=None), EINVAL),
    ({}, dict(T=-1), ESHAPE), ({}, dict(ldq=63), ESHAPE), ({}, dict(ldy=31), ESHAPE),
    ({}, dict(y=FAKE * 3 + 1), EINVAL), ({}, dict(dtype=F32, y=FAKE * 3 + 2), EINVAL), ({}, dict(q_scale=FAKE + 1), EINVAL),
    ({}, dict(y=FAKE + 16), EINVAL), ({}, dict(y=FAKE * 2 + 16), EINVAL), ({}, dict(y=FAKE * 100 + 16), EINVAL),
    ({}, dict(y=FAKE * 8000), EINVAL), ({"bias": FAKE * 3}, {}, EINVAL),
    ({"W": None}, {}, EINVAL), ({"scale": None}, {}, EINVAL), ({"bias": FAKE * 9 + 1}, {}, EINVAL),
    ({"scale": FAKE * 8000 + 2}, {}, EINVAL),
    ({"d_in": 0}, {}, ESHAPE), ({"d_out": 0}, {}, ESHAPE), ({"ldw": 63}, {}, ESHAPE), ({"ldw": 1 << 60}, {}, ESHAPE),
    ({"d_in": 131072, "ldw": 131072}, {}, EUNSUPPORTED),
])
def test_product_refusals(lib, w, kw, status):
    assert product(lib, weight(**w), **kw) == status


def test_product_without_weight(lib):
    assert lib.lora_base_product(None, FAKE, 64, FAKE * 2, 8, FAKE * 3, 32, BF16, None) == EINVAL


def apply(lib, w=None, **kw):
    v = dict(x=FAKE, ldx=64, T=8, y=FAKE * 3, ldy=32, dtype=BF16, ws=FAKE * 50, ws_bytes=1 << 16, stream=None)
    v.update(kw)
    w = weight() if w is None else w
    return lib.lora_base_apply(ctypes.addressof(w), *v.values())


@pytest.mark.parametrize("kw, status", [
    (dict(T=0, x=None, y=None, ws=None), 0),
    (dict(dtype=-1), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL),
    (dict(ws=None), EWORKSPACE), (dict(ws_bytes=767), EWORKSPACE), (dict(ws=FAKE * 50 + 8), EINVAL),
    (dict(T=-1), ESHAPE), (dict(ldx=63), ESHAPE), (dict(ldy=31), ESHAPE),
    (dict(x=FAKE + 1), EINVAL), (dict(y=FAKE + 1022), EINVAL), (dict(ws=FAKE), EINVAL), (dict(ws=FAKE * 3), EINVAL),
    (dict(ws=FAKE * 100), EINVAL), (dict(ws=FAKE * 8000), EINVAL),
])
def test_apply_refusals(lib, kw, status):
    assert apply(lib, **kw) == status


def test_workspace_size(lib):
    size = lambda w, n: lib.lora_base_workspace_size(ctypes.addressof(w), n)  # noqa: E731
    assert size(weight(), 0) == size(weight(), -1) == size(weight(d_in=0), 8) == 0
    for d_in in (1, 16, 17, 4096):
        w = weight(d_in=d_in, ldw=d_in)
        got = [size(w, n) for n in (1, 2, 7, 64, 65, 100000)]
        assert got == sorted(got)
        for n, b in zip((1, 2, 7, 64, 65, 100000), got):
            assert b >= n * (d_in + 4)
    # beyond 32 bits
    assert size(weight(d_in=14336, ldw=14336), 1 << 20) > 1 << 33


def heads(**kw):
    v = dict(src=FAKE * 4, dst=FAKE * 4, src_token=4 * 64, src_head=64, dst_token=4 * 64, dst_head=64, n_heads=4)
    v.update(kw)
    return v


def rotary(lib, slices=None, r=None, **kw):
    rr = dict(freq=FAKE * 200, head_dim=64, rot_dim=64, interleaved=0, mscale=1.0)
    rr.update(r or {})
    rr = L.lora_rotary(*rr.values())
    slices = [heads()] if slices is None else slices
    arr = (L.lora_rotary_slice * max(len(slices), 1))(*[L.lora_rotary_slice(*s.values()) for s in slices])
    v = dict(positions=FAKE, T=8, n=len(slices), array=ctypes.addressof(arr), dtype=BF16, inverse=0, stream=None)
    v.update(kw)
    return lib.lora_rotary_apply(ctypes.addressof(rr), *v.values())


@pytest.mark.parametrize("slices, r, kw, status", [
    (None, {}, dict(T=0, positions=None), 0),
    (None, {"freq": None}, {}, EINVAL), (None, {"freq": FAKE + 4}, {}, EINVAL), (None, {"interleaved": 2}, {}, EINVAL),
    (None, {}, dict(inverse=2), EINVAL), (None, {}, dict(dtype=3), EINVAL), (None, {}, dict(positions=None), EINVAL),
    (None, {}, dict(positions=FAKE + 2), EINVAL), (None, {}, dict(array=None), EINVAL),
    (None, {"rot_dim": 63}, {}, ESHAPE), (None, {"rot_dim": 66}, {}, ESHAPE), (None, {"rot_dim": 0}, {}, ESHAPE),
    (None, {"head_dim": 0}, {}, ESHAPE), (None, {"head_dim": 1026}, {}, EUNSUPPORTED),
    (None, {}, dict(T=-1), ESHAPE), (None, {}, dict(n=0), ESHAPE), ([heads()] * 9, {}, {}, ESHAPE),
    ([heads(src=None, dst=FAKE)], {}, {}, EINVAL), ([heads(dst=None)], {}, {}, EINVAL),
    ([heads(src=FAKE * 4 + 1, dst=FAKE * 4 + 1)], {}, {}, EINVAL),
    ([heads(n_heads=0)], {}, {}, ESHAPE), ([heads(dst_head=-64)], {}, {}, ESHAPE),
    ([heads(src_token=1 << 62)], {}, {}, ESHAPE),
    # values of dst that would share a place: a broadcast head, tokens that overlap
    ([heads(src=FAKE * 8, dst_head=0)], {}, {}, ESHAPE), ([heads(src=FAKE * 8, dst_token=200)], {}, {}, ESHAPE),
    # in place with other strides; a destination that meets the source
    ([heads(src_token=512)], {}, {}, ESHAPE), ([heads(dst=FAKE * 4 + 64)], {}, {}, EINVAL),
    # two slices that meet, in place and across
    ([heads(), heads()], {}, {}, EINVAL),
    ([heads(src=FAKE * 8), heads(src=FAKE * 4 + 128, dst=FAKE * 16)], {}, {}, EINVAL),
    # dst over the positions or the frequencies
    ([heads(dst=FAKE, src=FAKE * 8)], {}, {}, EINVAL), ([heads(dst=FAKE * 200, src=FAKE * 8)], {}, {}, EINVAL),
])
def test_rotary_refusals(lib, slices, r, kw, status):
    assert rotary(lib, slices, r, **kw) == status


def test_rotary_columns_that_meet_are_refused(lib):
    """Query and key heads as columns of one buffer, the key heads one value too early."""
    q = heads(src_token=6 * 64, dst_token=6 * 64)
    k = heads(src_token=6 * 64, dst_token=6 * 64, n_heads=2, src=FAKE * 4 + 4 * 128 - 2, dst=FAKE * 4 + 4 * 128 - 2)
    assert rotary(lib, [q, k]) == EINVAL


def test_frequencies():
    rot, base = 64, 10000.0
    j = np.arange(rot // 2)
    plain = base ** (-2.0 * j / rot)
    f = lambda **kw: L.lora_rotary_frequencies(rot, base, **kw).numpy()  # noqa: E731
    # pow is within an ulp of the true value on each side
    np.testing.assert_allclose(f(), plain, rtol=4 * 2.0 ** -52)
    np.testing.assert_allclose(f(scaling=L.LORA_ROTARY_LINEAR, factor=4.0), plain / 4, rtol=4 * 2.0 ** -52)
    b = f(scaling=L.LORA_ROTARY_BASE, factor=4.0)
    # ln of the raised base is off by some 2^-52 of 11, times an exponent below 1
    np.testing.assert_allclose(b[0], 1.0, rtol=0)
    np.testing.assert_allclose(b[-1], plain[-1] / 4, rtol=64 * 2.0 ** -52)
    p = f(scaling=L.LORA_ROTARY_PARTS, factor=8.0, length=8192.0, low=1.0, high=4.0)
    turns = 8192 * plain / (2 * math.pi)
    assert (turns > 4).any() and (turns < 1).any() and ((turns > 1) & (turns < 4)).any()
    keep = np.clip((turns - 1) / 3, 0, 1)
    np.testing.assert_allclose(p, keep * plain + (1 - keep) * plain / 8, rtol=64 * 2.0 ** -52)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=-2), dict(base=0.0), dict(base=math.inf), dict(base=math.nan),
    dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.0), dict(scaling=1, factor=math.nan),
    dict(scaling=2, rot_dim=2, factor=2.0), dict(scaling=3, factor=2.0, length=0.0, low=1.0, high=2.0),
    dict(scaling=3, factor=2.0, length=10.0, low=2.0, high=2.0), dict(scaling=3, factor=2.0, length=10.0, low=-1.0, high=2.0),
])
def test_frequency_refusals(kw):
    with pytest.raises(L.LoraError):
        L.lora_rotary_frequencies(**{"rot_dim": 8, **kw})


def test_host_tensors_are_refused():
    i8, f = torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(L.LoraError):
        L.BaseWeight(i8, f)
    with pytest.raises(L.LoraError):
        L.lora_quantize_rows(torch.zeros(2, 16), i8, f)
    with pytest.raises(L.LoraError):
        L.Rotary(torch.ones(4, dtype=torch.float64), 8)


class Stand:
    """What a call of the binding sees of a device tensor; its memory is never touched."""

    def __init__(self, dtype, *shape, strides=None):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda:0")
        n = [1]
        for s in shape[:0:-1]:
            n.insert(0, n[0] * s)
        self.strides = tuple(n) if strides is None else strides

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def get_device(self):
        return 0

    def data_ptr(self):
        return FAKE


@pytest.fixture
def launched(lib, monkeypatch):
    """The arguments of the calls that the binding would make, in place of the calls."""
    calls = []
    monkeypatch.setattr(L, "_launch", lambda index, what, f, *args: calls.append(args))
    return calls


MANY = (1 << 32) + 5


def stand_weight(d_out=8, d_in=4):
    return L.BaseWeight(Stand(torch.int8, d_out, d_in), Stand(torch.float32, d_out))


def stand_rotary():
    return L.Rotary(torch_freq(2), 4)


def torch_freq(n):
    f = Stand(torch.float64, n)
    f.numel = lambda: n
    return f


@pytest.mark.parametrize("call", [
    lambda: L.lora_quantize_rows(Stand(torch.float32, MANY, 4), Stand(torch.int8, MANY, 4), Stand(torch.float32, MANY)),
    lambda: L.lora_quantize_rows(Stand(torch.float32, 1, MANY), Stand(torch.int8, 1, MANY), Stand(torch.float32, 1)),
    lambda: L.lora_base_product(stand_weight(), Stand(torch.int8, MANY, 4), Stand(torch.float32, MANY),
                                Stand(torch.float32, MANY, 8)),
    lambda: L.lora_base_apply(stand_weight(), Stand(torch.float32, MANY, 4), Stand(torch.float32, MANY, 8),
                              Stand(torch.uint8, 1 << 40)),
    lambda: L.lora_rotary_apply(stand_rotary(), Stand(torch.int32, MANY), [Stand(torch.float32, MANY, 1, 4)]),
    lambda: L.lora_rotary_apply(stand_rotary(), Stand(torch.int32, 1), [Stand(torch.float32, 1, MANY, 4)]),
    lambda: stand_weight(d_out=MANY), lambda: stand_weight(d_in=MANY),
    lambda: L.lora_base_workspace_size(stand_weight(), MANY), lambda: L.new_base_workspace(stand_weight(), MANY),
    lambda: L.lora_rotary_frequencies(MANY + 1),
], ids=["quantize rows", "quantize columns", "product", "apply", "rotary tokens", "rotary heads", "weight rows",
        "weight columns", "workspace size", "workspace", "frequencies"])
def test_sizes_beyond_32_bits_are_refused(launched, call):
    """The C ABI's sizes are 32-bit: what does not fit is refused, not cut to its low bits."""
    with pytest.raises(L.LoraError):
        call()
    assert not launched


def one_row(dtype, n):
    """A tensor [1][n] as torch gives it for the transpose of a column: contiguous, with strides (1, 1)."""
    return Stand(dtype, 1, n, strides=(1, 1))


def test_one_row_may_have_any_row_stride(launched):
    """Where there is one row, its stride says nothing: the call gets one that fits its columns."""
    w = stand_weight(d_out=8, d_in=4)
    for x, y in ((one_row(torch.float32, 4), Stand(torch.float32, 1, 8)), (Stand(torch.float32, 1, 4), one_row(torch.float32, 8))):
        L.lora_base_apply(w, x, y, Stand(torch.uint8, 4096))
        ldx, ldy = launched[-1][2], launched[-1][5]
        assert ldx >= 4 and ldy >= 8
    for q, y in ((one_row(torch.int8, 4), Stand(torch.float32, 1, 8)), (Stand(torch.int8, 1, 4), one_row(torch.float32, 8))):
        L.lora_base_product(w, q, Stand(torch.float32, 1), y)
        ldq, ldy = launched[-1][2], launched[-1][6]
        assert ldq >= 4 and ldy >= 8
    for x, q in ((one_row(torch.float32, 4), Stand(torch.int8, 1, 4)), (Stand(torch.float32, 1, 4), one_row(torch.int8, 4))):
        L.lora_quantize_rows(x, q, Stand(torch.float32, 1))
        ldx, ldq = launched[-1][1], launched[-1][6]
        assert ldx >= 4 and ldq >= 4
    assert len(launched) == 6


def test_a_second_thread_never_sees_the_types_missing(monkeypatch):
    """At every bytecode of the binding's first look at torch: a thread that finds the module set finds its types too."""
    monkeypatch.setattr(L, "_torch_module", None)
    monkeypatch.setattr(L, "_REAL", {})
    seen = []

    def trace(frame, event, arg):
        if frame.f_code is L._torch.__code__:
            frame.f_trace_opcodes = True
            seen.append((L._torch_module is not None, len(L._REAL)))
            return trace
        return None

    old = sys.gettrace()
    sys.settrace(trace)
    try:
        L._torch()
    finally:
        sys.settrace(old)
    assert len(seen) > 5 and seen[0] == (False, 0) and seen[-1] == (True, 2)
    assert all(types == 2 for module, types in seen if module)


def product_kernels(lib, T, d_in, d_out):
    """The kernels that a product of rows of whole 16s takes, in turn, and the rows at which it is split."""
    first = ctypes.c_int32(-1)
    k = lib.lora_base_product_choice(T, d_in, d_out, ctypes.c_int64(d_in), ctypes.c_int64(d_in), ctypes.byref(first))
    if first.value == 0:
        return [k], []
    assert 0 < first.value < T
    (a, ra), (b, rb) = (product_kernels(lib, n, d_in, d_out) for n in (first.value, T - first.value))
    return a + b, [first.value, *ra, *(first.value + r for r in rb)]


def test_gpu_cases_take_every_kernel_of_the_product(lib):
    """Whatever costs the choice goes by: the sizes of the GPU tests take each tile shape, each kernel for few rows, each
    one for other rows, and splits of either large shape with different kernels for the rest."""
    import test_gpu_base as G
    assert {k for s in G.TILES for k in product_kernels(lib, *s)[0]} >= set(range(7)) | {11, 12}
    rest = set()
    for s in G.SPLITS:
        kernels, at = product_kernels(lib, *s)
        assert at, s
        rest.add((kernels[0], kernels[-1]))
    assert {a for a, _ in rest} == {0, 1} and len(rest) >= 4
    small = [(T, 512, 384) for T in (1, 17, 48)] + [(1, 17, 70), (100, 15, 70), (16, 65, 70)]
    assert {k for s in small for k in product_kernels(lib, *s)[0]} == {7, 8, 9, 10, 13}


def test_most_heads_of_a_slice(lib):
    """The limit on a slice's heads is the header's, and the binding's: one more is refused."""
    text = open(os.path.join(ROOT, "include", "lora_base.h")).read()
    most = int(re.search(r"#define\s+LORA_MAX_HEADS\s+(\d+)", text).group(1))
    assert most == L.LORA_MAX_HEADS
    assert re.search(r"int32_t n_heads;\s*/\*.*LORA_MAX_HEADS", text)
    wide = dict(src_token=(most + 1) * 64, dst_token=(most + 1) * 64)
    assert rotary(lib, [heads(n_heads=most + 1, **wide)], T=0) == ESHAPE
    assert rotary(lib, [heads(n_heads=most, **wide)], T=0) == 0
