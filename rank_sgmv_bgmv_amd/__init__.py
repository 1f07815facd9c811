"""Unmerged multi-LoRA (SGMV / BGMV) for AMD MI355X (gfx950).

A thin ctypes binding over the C-ABI library ``_build/liblora_hip.so``
(declared in ``include/lora.h``).  Every function here only marshals torch
tensors into pointers, sizes and the current HIP stream; every step of the
computation runs in the library's HIP kernels.  There is no CPU fallback: if
the library has not been built, calls raise ``LoraError``.

Functions carry the C names:
  lora_workspace_size, lora_plan_build, lora_apply, lora_apply_noalloc, lora_shrink, lora_expand,
  lora_apply_planned, lora_shrink_planned, lora_expand_planned,
  lora_apply_multi, lora_apply_sliced, lora_read_device_errors, lora_status_string,
  the operators around a LoRA layer (include/lora_base.h): lora_quantize_rows, lora_base_product, lora_base_apply,
  lora_base_workspace_size, lora_rotary_apply, lora_rotary_frequencies,
  and the measurement aids lora_calib_gather_read and lora_calib_tile_stream
  (include/lora_calib.h).

Tensors: A [n][r][d_in] and B [n][d_out][r] contiguous (float32 or bfloat16);
x [T][ldx], y [T][ldy] with unit column stride (ld = stride(0)); idx int32
[S][K]; seg_off int32 [S+1] or None (one token per request); scale float32
[S][K] or None; v float32 [T][ldv]; workspace/plan a uint8 device tensor.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

from . import accounting  # noqa: F401  (pure Python byte/FLOP accounting)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "liblora_hip.so")

LORA_F32, LORA_BF16 = 0, 1
STATUS = {0: "LORA_OK", -1: "LORA_EINVAL", -2: "LORA_ESHAPE", -3: "LORA_EWORKSPACE", -4: "LORA_EUNSUPPORTED",
          -5: "LORA_EHIP"}


class LoraError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = STATUS.get(status, str(status))
        super().__init__(f"{what}: {msg}" if what else msg)


class lora_pool(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("n_adapters", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("ranks", ctypes.c_void_p)]


class lora_batch(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("n_segments", ctypes.c_int32), ("seg_off", ctypes.c_void_p),
                ("idx", ctypes.c_void_p), ("max_slots", ctypes.c_int32), ("scale", ctypes.c_void_p)]


class lora_problem(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class lora_base_weight(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32)]


class lora_rotary(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float)]


class lora_rotary_slice(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("src_token", ctypes.c_int64),
                ("src_head", ctypes.c_int64), ("dst_token", ctypes.c_int64), ("dst_head", ctypes.c_int64),
                ("n_heads", ctypes.c_int32)]


_pack_slice = struct.Struct("@PPqqqqi4x").pack  # a lora_rotary_slice's bytes

LORA_ROTARY_PLAIN, LORA_ROTARY_LINEAR, LORA_ROTARY_BASE, LORA_ROTARY_PARTS = 0, 1, 2, 3
LORA_MAX_SLICES, LORA_MAX_HEADS = 8, 65535

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises LoraError if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LoraError(-5, f"HIP library not built ({LIB_PATH}); run python -m rank_sgmv_bgmv_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        pp, pb = ctypes.POINTER(lora_pool), ctypes.POINTER(lora_batch)
        sig = {
            "lora_workspace_size": (SZ, [pb, I32]),
            "lora_plan_build": (ctypes.c_int, [pb, I32, P, SZ, P]),
            "lora_apply": (ctypes.c_int, [pp, pb, P, I64, P, I64, P, SZ, P]),
            "lora_apply_noalloc": (ctypes.c_int, [pp, pb, P, I64, P, I64, P]),
            "lora_shrink": (ctypes.c_int, [pp, pb, P, I64, P, I64, P, SZ, P]),
            "lora_expand": (ctypes.c_int, [pp, pb, P, I64, P, I64, P, SZ, P]),
            "lora_apply_planned": (ctypes.c_int, [pp, pb, P, SZ, P, I64, P, I64, P]),
            "lora_shrink_planned": (ctypes.c_int, [pp, pb, P, SZ, P, I64, P, I64, P]),
            "lora_expand_planned": (ctypes.c_int, [pp, pb, P, SZ, P, I64, P, I64, P]),
            "lora_apply_multi": (ctypes.c_int, [pp, pb, P, SZ, I32, P, I32, P]),
            "lora_apply_sliced": (ctypes.c_int, [pp, pb, P, SZ, I32, I32, P, P, I32, P]),
            "lora_read_device_errors": (ctypes.c_int, [P, SZ, ctypes.POINTER(I32), P]),
            "lora_merge": (ctypes.c_int, [pp, P, P, I32, ctypes.c_float, P, I64, P]),
            "lora_merge_multi": (ctypes.c_int, [pp, P, P, I32, ctypes.c_float, I32, P, I32, P]),
            "lora_pool_load": (ctypes.c_int, [pp, I32, P, P, P]),
            "lora_calib_gather_read": (ctypes.c_int, [P, P, I32, I32, I32, P, I32, I32, P, P]),
            "lora_calib_tile_stream": (ctypes.c_int, [P, P, I32, I32, I32, P, I32, I32, I32, P, P]),
            "lora_quantize_rows": (ctypes.c_int, [P, I64, ctypes.c_int, I32, I32, P, I64, P, P]),
            "lora_base_product": (ctypes.c_int, [P, P, I64, P, I32, P, I64, ctypes.c_int, P]),
            "lora_base_workspace_size": (SZ, [P, I32]),
            "lora_base_apply": (ctypes.c_int, [P, P, I64, I32, P, I64, ctypes.c_int, P, SZ, P]),
            "lora_rotary_apply": (ctypes.c_int, [P, P, I32, I32, P, ctypes.c_int, I32, P]),
            "lora_rotary_frequencies": (ctypes.c_int, [ctypes.c_int, ctypes.c_double, I32] + [ctypes.c_double] * 4 + [P]),
            "lora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "lora_abi_version": (I32, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


# ------------------------------------------------------------- marshalling --
def _torch():
    global _torch_module, _REAL
    if _torch_module is None:
        import torch
        _REAL = {torch.bfloat16: LORA_BF16, torch.float32: LORA_F32}
        _torch_module = torch  # last: who finds it, in another thread too, finds the types
    return _torch_module


_torch_module, _REAL = None, {}


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return LORA_F32
    if t.dtype == torch.bfloat16:
        return LORA_BF16
    raise LoraError(-1, f"unsupported dtype {t.dtype}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(t) -> int:
    torch = _torch()
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(st: int, what: str):
    if st != 0:
        raise LoraError(st, what)


class Pool:
    """A resident adapter pool: A [n][r][d_in], B [n][d_out][r]; ranks: an optional
    int32 device tensor [n] of per-adapter ranks (adapters stored at rank r)."""

    def __init__(self, A, B, ranks=None):
        if A.dim() != 3 or B.dim() != 3 or not A.is_contiguous() or not B.is_contiguous():
            raise LoraError(-2, "A and B must be contiguous 3-D tensors")
        n, r, d_in = A.shape
        if B.shape[0] != n or B.shape[2] != r or B.dtype != A.dtype:
            raise LoraError(-2, "B must be [n][d_out][r] with A's dtype")
        if ranks is not None and (ranks.dtype != _torch().int32 or tuple(ranks.shape) != (n,)
                                  or not ranks.is_contiguous() or ranks.device != A.device):
            raise LoraError(-2, "ranks must be a contiguous int32 device tensor [n]")
        self.A, self.B, self.ranks = A, B, ranks
        self.n, self.r, self.d_in, self.d_out = int(n), int(r), int(d_in), int(B.shape[1])
        self.c = lora_pool(_ptr(A), _ptr(B), self.n, self.r, self.d_in, self.d_out, _dtype_code(A), _ptr(ranks))


class Batch:
    """Which adapters apply to which rows (see lora_batch in include/lora.h)."""

    def __init__(self, n_tokens: int, idx, seg_off=None, scale=None):
        torch = _torch()
        if idx.dtype != torch.int32 or idx.dim() != 2 or not idx.is_contiguous():
            raise LoraError(-2, "idx must be a contiguous int32 [S][K] tensor")
        S, K = idx.shape
        if seg_off is not None and (seg_off.dtype != torch.int32 or seg_off.numel() != S + 1):
            raise LoraError(-2, "seg_off must be int32 [S+1]")
        if scale is not None and (scale.dtype != torch.float32 or tuple(scale.shape) != (S, K)
                                  or not scale.is_contiguous()):
            raise LoraError(-2, "scale must be a contiguous float32 [S][K] tensor")
        if seg_off is None and S != n_tokens:
            raise LoraError(-2, "per-token mode needs idx with n_tokens rows")
        self.idx, self.seg_off, self.scale = idx, seg_off, scale
        self.T, self.S, self.K = int(n_tokens), int(S), int(K)
        self.c = lora_batch(self.T, self.S, _ptr(seg_off), _ptr(idx), self.K, _ptr(scale))


def _ld(t) -> int:
    if t.dim() != 2:
        raise LoraError(-2, "activations must be 2-D")
    if t.numel() == 0:  # no rows: torch reports arbitrary strides for empty views
        return max(int(t.shape[1]), 1)
    if t.stride(1) != 1:
        raise LoraError(-2, "activations must have unit column stride")
    return int(t.stride(0))


def _same_device(what: str, dev, *tensors):
    for t in tensors:
        if t is not None and t.device != dev:
            raise LoraError(-1, f"{what}: every tensor must be on {dev} (found {t.device})")


def _check_rows(what: str, pool: "Pool", batch: Batch, x=None, y=None, v=None, ws=None):
    """Shapes, dtypes and devices of one call's tensors against its pool and batch:
    x [>= T][>= d_in] and y [>= T][>= d_out] of the pool's dtype, v float32
    [>= T][>= K*r], everything (batch tensors included) on the pool's device."""
    torch = _torch()
    dev = pool.A.device
    if dev.type != "cuda":
        raise LoraError(-1, f"{what}: the pool must be in device memory")
    _same_device(what, dev, pool.B, pool.ranks, batch.idx, batch.seg_off, batch.scale, x, y, v, ws)
    for name, t, cols, dt in (("x", x, pool.d_in, pool.A.dtype), ("y", y, pool.d_out, pool.A.dtype),
                              ("v", v, batch.K * pool.r, torch.float32)):
        if t is None:
            continue
        if t.dim() != 2 or t.shape[0] < batch.T or t.shape[1] < cols:
            raise LoraError(-2, f"{what}: {name} must be at least [{batch.T}][{cols}] (got {tuple(t.shape)})")
        if t.dtype != dt:
            raise LoraError(-2, f"{what}: {name} must be {dt} (got {t.dtype})")


def lora_workspace_size(batch: Batch, n_adapters: int) -> int:
    return int(lib().lora_workspace_size(ctypes.byref(batch.c), n_adapters))


def new_workspace(batch: Batch, n_adapters: int, device):
    torch = _torch()
    nbytes = lora_workspace_size(batch, n_adapters)
    if nbytes == 0:
        raise LoraError(-2, "invalid batch")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def lora_plan_build(batch: Batch, n_adapters: int, plan):
    _same_device("lora_plan_build", plan.device, batch.idx, batch.seg_off, batch.scale)
    _check(lib().lora_plan_build(ctypes.byref(batch.c), n_adapters, _ptr(plan), plan.numel(), _stream(plan)),
           "lora_plan_build")


def lora_apply(pool: Pool, batch: Batch, x, y, ws):
    _check_rows("lora_apply", pool, batch, x=x, y=y, ws=ws)
    _check(lib().lora_apply(ctypes.byref(pool.c), ctypes.byref(batch.c), _ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(ws),
                            ws.numel(), _stream(y)), "lora_apply")


def lora_apply_noalloc(pool: Pool, batch: Batch, x, y):
    """lora_apply with the plan in the library's own device array (no workspace,
    nothing allocated); calls that overlap on one GPU race."""
    _check_rows("lora_apply_noalloc", pool, batch, x=x, y=y)
    _check(lib().lora_apply_noalloc(ctypes.byref(pool.c), ctypes.byref(batch.c), _ptr(x), _ld(x), _ptr(y), _ld(y),
                                    _stream(y)), "lora_apply_noalloc")


def lora_shrink(pool: Pool, batch: Batch, x, v, ws):
    _check_rows("lora_shrink", pool, batch, x=x, v=v, ws=ws)
    _check(lib().lora_shrink(ctypes.byref(pool.c), ctypes.byref(batch.c), _ptr(x), _ld(x), _ptr(v), _ld(v),
                             _ptr(ws), ws.numel(), _stream(v)), "lora_shrink")


def lora_expand(pool: Pool, batch: Batch, v, y, ws):
    _check_rows("lora_expand", pool, batch, y=y, v=v, ws=ws)
    _check(lib().lora_expand(ctypes.byref(pool.c), ctypes.byref(batch.c), _ptr(v), _ld(v), _ptr(y), _ld(y),
                             _ptr(ws), ws.numel(), _stream(y)), "lora_expand")


def lora_apply_planned(pool: Pool, batch: Batch, plan, x, y):
    _check_rows("lora_apply_planned", pool, batch, x=x, y=y, ws=plan)
    _check(lib().lora_apply_planned(ctypes.byref(pool.c), ctypes.byref(batch.c), _ptr(plan), plan.numel(), _ptr(x),
                                    _ld(x), _ptr(y), _ld(y), _stream(y)), "lora_apply_planned")


def lora_shrink_planned(pool: Pool, batch: Batch, plan, x, v):
    _check_rows("lora_shrink_planned", pool, batch, x=x, v=v, ws=plan)
    _check(lib().lora_shrink_planned(ctypes.byref(pool.c), ctypes.byref(batch.c), _ptr(plan), plan.numel(), _ptr(x),
                                     _ld(x), _ptr(v), _ld(v), _stream(v)), "lora_shrink_planned")


def lora_expand_planned(pool: Pool, batch: Batch, plan, v, y):
    _check_rows("lora_expand_planned", pool, batch, y=y, v=v, ws=plan)
    _check(lib().lora_expand_planned(ctypes.byref(pool.c), ctypes.byref(batch.c), _ptr(plan), plan.numel(), _ptr(v),
                                     _ld(v), _ptr(y), _ld(y), _stream(y)), "lora_expand_planned")


def problems_table(problems: Sequence, device):
    """Device array of lora_problem for (A, B, x, y) tuples of one shape; returns
    (table tensor, all_aligned).  The tensors must stay alive while it is used."""
    torch = _torch()
    rows, aligned = [], True
    for A, B, x, y in problems:
        e = 8 if A.dtype == torch.bfloat16 else 4
        ldx, ldy = _ld(x), _ld(y)
        ptrs = [_ptr(A), _ptr(B), _ptr(x), _ptr(y)]
        aligned &= all(p % 16 == 0 for p in ptrs) and ldx % e == 0 and ldy % e == 0
        rows.append(ptrs + [ldx, ldy])
    table = torch.tensor(rows, dtype=torch.int64).to(device)
    return table, aligned


def lora_apply_multi(shape: Pool, batch: Batch, plan, table, aligned: bool = True):
    """shape: a Pool whose shape (n, r, d_in, d_out, dtype) all problems share."""
    n = int(table.shape[0]) if table.numel() else 0
    _check_rows("lora_apply_multi", shape, batch, ws=plan)
    _same_device("lora_apply_multi", plan.device, table)
    _check(lib().lora_apply_multi(ctypes.byref(shape.c), ctypes.byref(batch.c), _ptr(plan), plan.numel(), n,
                                  _ptr(table), 1 if aligned else 0, _stream(plan)), "lora_apply_multi")


def sliced_table(groups: Sequence, device):
    """Device array of lora_problem for lora_apply_sliced.  groups: a sequence of
    (x, [(A, B, y), ...]) -- one x and its slices (the same number of slices, of
    the same output widths, in every group).  Returns (table, d_outs, all_aligned).
    The tensors must stay alive while the table is used."""
    rows, d_outs = [], None
    for x, slices in groups:
        widths = [int(B.shape[1]) for _, B, _ in slices]
        if d_outs is None:
            d_outs = widths
        elif widths != d_outs:
            raise LoraError(-2, "every group must have slices of the same output widths")
        rows += [(A, B, x, y) for A, B, y in slices]
    table, aligned = problems_table(rows, device)
    return table, d_outs or [], aligned


def lora_apply_sliced(shape: Pool, batch: Batch, plan, table, d_outs: Sequence[int], aligned: bool = True):
    """Groups of projections that read one x (q / k / v, gate / up), one launch:
    table from sliced_table; shape gives n, rank, d_in, dtype (and ranks)."""
    ns = len(d_outs)
    rows = int(table.shape[0]) if table.numel() else 0
    if ns < 1 or rows % ns:
        raise LoraError(-2, "table rows must be a whole number of groups of len(d_outs) slices")
    widths = (ctypes.c_int32 * ns)(*[int(v) for v in d_outs])
    _check_rows("lora_apply_sliced", shape, batch, ws=plan)
    _same_device("lora_apply_sliced", plan.device, table)
    _check(lib().lora_apply_sliced(ctypes.byref(shape.c), ctypes.byref(batch.c), _ptr(plan), plan.numel(), rows // ns,
                                   ns, widths, _ptr(table), 1 if aligned else 0, _stream(plan)), "lora_apply_sliced")


def lora_merge(pool: Pool, idx: Sequence[int], W, scale: Optional[Sequence[float]] = None, alpha: float = 1.0):
    """W += alpha * sum_k scale[k] B_idx[k] A_idx[k] in place (alpha = -1 unmerges).
    idx and scale are host sequences; W is a [d_out][ldw] device tensor of the pool's dtype."""
    if W.dim() != 2 or W.shape[0] != pool.d_out or W.shape[1] < pool.d_in or W.dtype != pool.A.dtype:
        raise LoraError(-2, "W must be [d_out][>= d_in] with the pool's dtype")
    ids = (ctypes.c_int32 * len(idx))(*[int(i) for i in idx])
    sc = None if scale is None else (ctypes.c_float * len(scale))(*[float(v) for v in scale])
    _check(lib().lora_merge(ctypes.byref(pool.c), ids, sc, len(idx), float(alpha), _ptr(W), _ld(W), _stream(W)),
           "lora_merge")


def merge_table(problems: Sequence, device):
    """Device array of lora_merge_problem for (A, B, W) tuples of one shape;
    returns (table tensor, all_aligned).  The tensors must stay alive while it is used."""
    torch = _torch()
    rows, aligned = [], True
    for A, B, W in problems:
        e = 8 if A.dtype == torch.bfloat16 else 4
        ldw = _ld(W)
        ptrs = [_ptr(A), _ptr(B), _ptr(W)]
        aligned &= all(p % 16 == 0 for p in ptrs) and ldw % e == 0
        rows.append(ptrs + [ldw])
    table = torch.tensor(rows, dtype=torch.int64).to(device)
    return table, aligned


def lora_merge_multi(shape: Pool, idx: Sequence[int], table, aligned: bool = True,
                     scale: Optional[Sequence[float]] = None, alpha: float = 1.0):
    """lora_merge over every (A, B, W) of a merge_table in one launch."""
    ids = (ctypes.c_int32 * len(idx))(*[int(i) for i in idx])
    sc = None if scale is None else (ctypes.c_float * len(scale))(*[float(v) for v in scale])
    n = int(table.shape[0]) if table.numel() else 0
    _check(lib().lora_merge_multi(ctypes.byref(shape.c), ids, sc, len(idx), float(alpha), n, _ptr(table),
                                  1 if aligned else 0, _stream(table)), "lora_merge_multi")


def lora_pool_load(pool: Pool, slot: int, A_host, B_host, stream=None):
    """Copy one adapter (host tensors [r][d_in] and [d_out][r], the pool's dtype,
    contiguous; pinned for an asynchronous copy) into slot `slot` of the pool,
    on `stream` (a torch.cuda.Stream; the current stream by default)."""
    torch = _torch()
    if A_host.device.type != "cpu" or B_host.device.type != "cpu":
        raise LoraError(-1, "A_host and B_host must be host tensors")
    if (tuple(A_host.shape) != (pool.r, pool.d_in) or tuple(B_host.shape) != (pool.d_out, pool.r)
            or not A_host.is_contiguous() or not B_host.is_contiguous()
            or A_host.dtype != pool.A.dtype or B_host.dtype != pool.A.dtype):
        raise LoraError(-2, "A_host must be [r][d_in] and B_host [d_out][r], contiguous, of the pool's dtype")
    s = (stream or torch.cuda.current_stream(pool.A.device)).cuda_stream
    _check(lib().lora_pool_load(ctypes.byref(pool.c), int(slot), _ptr(A_host), _ptr(B_host), s), "lora_pool_load")


# ------------------------------------------- around a LoRA layer (lora_base.h) --
# A decode step's kernels take a few microseconds, as does a call's way through
# Python: these bindings look first for tensors that are plainly right (_row,
# _line), and where one is not go through the checks that name what is wrong.
def _launch(index: int, what: str, f, *args):
    """f(*args, stream) on the current stream of device `index`, as the current device: launches go to that one."""
    C = _torch()._C
    if index == C._cuda_getDevice():
        st = f(*args, C._cuda_getCurrentRawStream(index))
    else:
        with _torch().cuda.device(index):
            st = f(*args, C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise LoraError(st, what)


_INT32_MAX = 0x7fffffff


def _fits_32(what: str, a: int, b: int = 0):
    """The C ABI's sizes are 32-bit; the call would get the low bits of a larger one."""
    if a > _INT32_MAX or b > _INT32_MAX:
        raise LoraError(-2, f"{what}: sizes must be below 2^31 (got {max(a, b)})")


def _row(t, dtype, index: int) -> int:
    """The row stride of a 2-D tensor of this type and device with unit column stride; 0 if t is not plainly one.
    (One below the columns is not plain either: a single row may have any.)"""
    if t.dtype is not dtype or t.get_device() != index:
        return 0
    s = t.stride()
    return s[0] if len(s) == 2 and s[1] == 1 else 0


def _line(t, dtype, index: int, n: int) -> bool:
    """Whether t is plainly a contiguous 1-D tensor of n elements or more, of this type and device."""
    return t.dtype is dtype and t.get_device() == index and t.stride() == (1,) and t.shape[0] >= n


def _rows_2d(what: str, name: str, t, dtypes, dev, cols: int, rows: Optional[int] = None) -> int:
    """Checks one 2-D tensor of a call and returns its row stride."""
    if t.device != dev or dev.type != "cuda":
        raise LoraError(-1, f"{what}: {name} must be in device memory, every tensor on {dev} (found {t.device})")
    if t.dtype not in dtypes:
        raise LoraError(-2, f"{what}: {name} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    if t.dim() != 2 or t.shape[1] < cols or (rows is not None and t.shape[0] < rows):
        raise LoraError(-2, f"{what}: {name} must be at least [{'*' if rows is None else rows}][{cols}] "
                            f"(got {tuple(t.shape)})")
    if t.shape[0] == 0:
        return max(int(t.shape[1]), 1)
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise LoraError(-2, f"{what}: {name} must have unit column stride")
    if t.shape[0] == 1:
        return int(t.shape[1])
    return int(t.stride(0))


def _vector(what: str, name: str, t, dtype, dev, n: int):
    if t.device != dev or t.dtype != dtype or t.dim() != 1 or t.shape[0] < n or (n > 1 and t.stride(0) != 1):
        raise LoraError(-2, f"{what}: {name} must be {dtype} [{n}] on {dev}, contiguous")


class BaseWeight:
    """A base weight in 8 bits (lora_base_weight): W int8 [d_out][d_in] (unit column stride), scale float32 [d_out],
    bias float32 [d_out] or None.  Keeps the tensors alive."""

    def __init__(self, W, scale, bias=None):
        torch = _torch()
        if W.dim() != 2 or W.shape[0] < 1 or W.shape[1] < 1:
            raise LoraError(-2, "W must be [d_out][d_in]")
        self.ld = _rows_2d("BaseWeight", "W", W, (torch.int8,), W.device, 1)
        self.d_out, self.d_in = int(W.shape[0]), int(W.shape[1])
        _fits_32("BaseWeight", self.d_out, self.d_in)
        for name, t in (("scale", scale), ("bias", bias)):
            if t is not None:
                _vector("BaseWeight", name, t, torch.float32, W.device, self.d_out)
                if t.shape[0] != self.d_out:
                    raise LoraError(-2, f"BaseWeight: {name} must be [{self.d_out}]")
        self.W, self.scale, self.bias, self.device = W, scale, bias, W.device
        self.c = lora_base_weight(_ptr(W), _ptr(scale), _ptr(bias), self.ld, self.d_in, self.d_out)
        self.ref, self.index = ctypes.addressof(self.c), W.get_device()


def lora_quantize_rows(x, q, scale):
    """q[t] = rint(127 x[t] / max|x[t]|) and scale[t] = max|x[t]| / 127 for every row of x [T][d]
    (bfloat16 or float32) into q int8 [T][d] and scale float32 [T]."""
    torch = _torch()
    what, index = "lora_quantize_rows", x.get_device()
    code = _REAL.get(x.dtype, -1)
    ldx, ldq = _row(x, x.dtype, index), _row(q, torch.int8, index)
    T, d = x.shape if ldx else (0, 0)
    if (index < 0 or code < 0 or ldx == 0 or ldx < d or ldq == 0 or ldq < d or q.shape != (T, d) or T > _INT32_MAX
            or d > _INT32_MAX or not _line(scale, torch.float32, index, T)):
        dev = x.device
        if x.dim() != 2 or q.dim() != 2 or x.shape != q.shape:
            raise LoraError(-2, f"{what}: x and q must be of one shape [T][d]")
        ldx = _rows_2d(what, "x", x, _REAL, dev, 1)
        ldq = _rows_2d(what, "q", q, (torch.int8,), dev, 1)
        T, d = x.shape
        _vector(what, "scale", scale, torch.float32, dev, T)
        _fits_32(what, T, d)
    _launch(index, what, lib().lora_quantize_rows, x.data_ptr(), ldx, code, T, d, q.data_ptr(), ldq, scale.data_ptr())


def lora_base_product(weight: BaseWeight, q, q_scale, y):
    """y[t][o] = q_scale[t] scale[o] sum_c q[t][c] W[o][c] (+ bias[o]) for every row of q int8 [T][d_in] into
    y [T][>= d_out] (bfloat16 or float32; further rows and columns are left as they are)."""
    torch = _torch()
    what, index, d_in = "lora_base_product", weight.index, weight.d_in
    code = _REAL.get(y.dtype, -1)
    ldq, ldy = _row(q, torch.int8, index), _row(y, y.dtype, index)
    T = q.shape[0] if ldq else 0
    if (code < 0 or ldq < d_in or ldy < weight.d_out or q.shape[1] != d_in or y.shape[0] < T or y.shape[1] < weight.d_out
            or T > _INT32_MAX or not _line(q_scale, torch.float32, index, T)):
        dev = weight.device
        ldq = _rows_2d(what, "q", q, (torch.int8,), dev, d_in)
        T = q.shape[0]
        if q.shape[1] != d_in:
            raise LoraError(-2, f"{what}: q must be [T][{d_in}]")
        ldy = _rows_2d(what, "y", y, _REAL, dev, weight.d_out, T)
        _vector(what, "q_scale", q_scale, torch.float32, dev, T)
        _fits_32(what, T)
    _launch(index, what, lib().lora_base_product, weight.ref, q.data_ptr(), ldq, q_scale.data_ptr(), T, y.data_ptr(), ldy,
            code)


def lora_base_workspace_size(weight: BaseWeight, n_tokens: int) -> int:
    _fits_32("lora_base_workspace_size", n_tokens)
    return int(lib().lora_base_workspace_size(weight.ref, max(n_tokens, 0)))


def new_base_workspace(weight: BaseWeight, n_tokens: int):
    """A workspace for lora_base_apply on up to n_tokens rows of this weight."""
    return _torch().empty(max(lora_base_workspace_size(weight, n_tokens), 16), dtype=_torch().uint8, device=weight.device)


def lora_base_apply(weight: BaseWeight, x, y, ws):
    """lora_quantize_rows and lora_base_product in one call: y [T][>= d_out] from x [T][d_in] of the same type, the
    quantised rows in the uint8 workspace ws (new_base_workspace)."""
    torch = _torch()
    what, index, d_in = "lora_base_apply", weight.index, weight.d_in
    code = _REAL.get(x.dtype, -1)
    ldx, ldy = _row(x, x.dtype, index), _row(y, x.dtype, index)
    T = x.shape[0] if ldx else 0
    if (code < 0 or ldx < d_in or ldy < weight.d_out or x.shape[1] != d_in or y.shape[0] < T or y.shape[1] < weight.d_out
            or T > _INT32_MAX or not _line(ws, torch.uint8, index, 0)):
        dev = weight.device
        ldx = _rows_2d(what, "x", x, _REAL, dev, d_in)
        T = x.shape[0]
        if x.shape[1] != d_in:
            raise LoraError(-2, f"{what}: x must be [T][{d_in}]")
        ldy = _rows_2d(what, "y", y, (x.dtype,), dev, weight.d_out, T)
        _vector(what, "ws", ws, torch.uint8, dev, 0)
        _fits_32(what, T)
    _launch(index, what, lib().lora_base_apply, weight.ref, x.data_ptr(), ldx, T, y.data_ptr(), ldy, code, ws.data_ptr(),
            ws.shape[0])


class Rotary:
    """Rotary positions of one model (lora_rotary): freq float64 [rot_dim / 2] on the device, radians per position
    (lora_rotary_frequencies), the heads' size, which values are pairs, and a factor of the rotated ones."""

    def __init__(self, freq, head_dim: int, interleaved: bool = False, mscale: float = 1.0):
        if freq.device.type != "cuda":
            raise LoraError(-1, "Rotary: freq must be in device memory")
        if freq.numel() < 1 or 2 * freq.numel() > head_dim:
            raise LoraError(-2, "Rotary: freq must be [rot_dim / 2] with rot_dim <= head_dim")
        _vector("Rotary", "freq", freq, _torch().float64, freq.device, freq.numel())
        self.freq, self.device, self.head_dim = freq, freq.device, int(head_dim)
        self.c = lora_rotary(_ptr(freq), self.head_dim, 2 * freq.numel(), int(bool(interleaved)), float(mscale))
        self.ref, self.index = ctypes.addressof(self.c), freq.get_device()


def lora_rotary_apply(rotary: Rotary, positions, src: Sequence, dst: Optional[Sequence] = None, inverse: bool = False):
    """Rotates the heads of src, up to 8 tensors [T][heads][head_dim] of the same tokens (any token and head
    strides, 1 to LORA_MAX_HEADS heads), into dst (in place by default).  positions int32 [T]; tokens of a negative position are skipped."""
    torch = _torch()
    what, index, D = "lora_rotary_apply", rotary.index, rotary.head_dim
    n, T = len(src), positions.shape[0] if positions.dim() else 0
    if not 1 <= n <= LORA_MAX_SLICES or (dst is not None and len(dst) != n):
        raise LoraError(-2, f"{what}: 1 to {LORA_MAX_SLICES} tensors, as many in dst as in src")
    if T > _INT32_MAX or not _line(positions, torch.int32, index, T):
        _vector(what, "positions", positions, torch.int32, rotary.device, T)
        _fits_32(what, T)
    dtype = src[0].dtype
    code = _REAL.get(dtype, -1)
    if code < 0:
        raise LoraError(-2, f"{what}: heads must be bfloat16 or float32 (got {dtype})")
    slices = b""
    for i in range(n):
        a = src[i]
        shape, sa, pa = a.shape, a.stride(), a.data_ptr()
        if a.dtype is not dtype or a.get_device() != index or len(shape) != 3 or shape[0] != T or shape[2] != D or (
                sa[2] != 1 and D > 1):
            raise LoraError(-2, f"{what}: heads must be {dtype} [{T}][heads][{D}] on {rotary.device}, a head's values "
                                f"side by side (got {a.dtype} {tuple(shape)} on {a.device}, strides {sa})")
        sb, pb = sa, pa
        if dst is not None:
            b = dst[i]
            sb, pb = b.stride(), b.data_ptr()
            if b.dtype is not dtype or b.get_device() != index or b.shape != shape or (sb[2] != 1 and D > 1):
                raise LoraError(-2, f"{what}: dst must be like src (got {b.dtype} {tuple(b.shape)} on {b.device}, "
                                    f"strides {sb})")
        if shape[1] > _INT32_MAX:
            _fits_32(what, shape[1])
        slices += _pack_slice(pa, pb, sa[0], sa[1], sb[0], sb[1], shape[1])
    _launch(index, what, lib().lora_rotary_apply, rotary.ref, positions.data_ptr(), T, n, slices, code, 1 if inverse else 0)


def lora_rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: int = LORA_ROTARY_PLAIN, factor: float = 1.0,
                            length: float = 1.0, low: float = 0.0, high: float = 1.0):
    """Frequencies float64 [rot_dim / 2] on the host (include/lora_base.h: the scalings of long contexts)."""
    _fits_32("lora_rotary_frequencies", rot_dim)
    freq = _torch().empty(max(int(rot_dim), 0) // 2, dtype=_torch().float64)
    _check(lib().lora_rotary_frequencies(int(scaling), float(base), int(rot_dim), float(factor), float(length),
                                         float(low), float(high), _ptr(freq) if freq.numel() else None),
           "lora_rotary_frequencies")
    return freq


def lora_read_device_errors(plan) -> int:
    cnt = ctypes.c_int32(0)
    _check(lib().lora_read_device_errors(_ptr(plan), plan.numel(), ctypes.byref(cnt), _stream(plan)),
           "lora_read_device_errors")
    return int(cnt.value)


def lora_status_string(status: int) -> str:
    return lib().lora_status_string(status).decode()


def plan_header(plan):
    """The plan's header words (a host copy; synchronizes)."""
    return plan[:256].view(_torch().int32).cpu().tolist()[:16]


def lora_calib_gather_read(pool, off, blocks_per_group: int, block_bytes: int, sink, rmw=None, rmw_bytes: int = 0,
                           lds_bytes: int = 0):
    """Measurement aid (include/lora_calib.h): workgroup g reads the
    blocks_per_group blocks of `pool` (a device tensor) that start at byte
    offsets off[g * blocks_per_group ...] (int64 device tensor), block_bytes
    each; with `rmw` it also reads and writes back rmw_bytes of rmw at
    g * rmw_bytes.  Each workgroup reserves lds_bytes of LDS it does not use
    (limiting how many share a compute unit).  sink (int32 device tensor, one
    word per group) receives each group's XOR.  The caller keeps every block
    inside `pool`."""
    torch = _torch()
    if off.dtype != torch.int64 or blocks_per_group < 1 or off.numel() % blocks_per_group:
        raise LoraError(-2, "lora_calib_gather_read: off must be int64, blocks_per_group offsets per group")
    n_groups = off.numel() // blocks_per_group
    if sink.numel() * sink.element_size() < 4 * n_groups:
        raise LoraError(-2, "lora_calib_gather_read: sink must hold one word per group")
    if rmw is not None and rmw.numel() * rmw.element_size() < n_groups * rmw_bytes:
        raise LoraError(-2, "lora_calib_gather_read: rmw must hold rmw_bytes per group")
    _same_device("lora_calib_gather_read", pool.device, off, sink, rmw)
    _check(lib().lora_calib_gather_read(_ptr(pool), _ptr(off), n_groups, blocks_per_group, block_bytes, _ptr(rmw),
                                        rmw_bytes if rmw is not None else 0, lds_bytes, _ptr(sink), _stream(pool)),
           "lora_calib_gather_read")


def lora_calib_tile_stream(x, y, rows: int, row_bytes: int, sink, order: int = 0, adapters=None,
                           n_adapters: int = 0, lds_bytes: int = 0):
    """Measurement aid (include/lora_calib.h): the prefill tiles' traffic with
    no arithmetic.  Workgroup t reads its `rows` rows (row_bytes each) of the
    device tensors x and y and writes y's back unchanged, in the MFMA
    kernel's stage order (order 0, reading a stage of adapter t % n_adapters
    beside each when `adapters` is given) or whole rows at a time (order 1).
    sink (int32 device tensor, one word per tile) receives each tile's XOR."""
    if rows < 1 or row_bytes < 1 or x.numel() * x.element_size() % (rows * row_bytes):
        raise LoraError(-2, "lora_calib_tile_stream: x must hold whole tiles of rows x row_bytes")
    n_tiles = x.numel() * x.element_size() // (rows * row_bytes)
    if y.numel() * y.element_size() != x.numel() * x.element_size():
        raise LoraError(-2, "lora_calib_tile_stream: y must be the size of x")
    if sink.numel() * sink.element_size() < 4 * n_tiles:
        raise LoraError(-2, "lora_calib_tile_stream: sink must hold one word per tile")
    if adapters is not None:
        per = row_bytes // 512 * 32768 + row_bytes // 256 * 16384
        if n_adapters < 1 or adapters.numel() * adapters.element_size() < n_adapters * per:
            raise LoraError(-2, "lora_calib_tile_stream: adapters must hold n_adapters A and B blocks")
    _same_device("lora_calib_tile_stream", x.device, y, sink, adapters)
    _check(lib().lora_calib_tile_stream(_ptr(x), _ptr(y), n_tiles, rows, row_bytes, _ptr(adapters),
                                        n_adapters if adapters is not None else 0, order, lds_bytes, _ptr(sink),
                                        _stream(x)),
           "lora_calib_tile_stream")
