"""The many-token operators of the binding: the MACKO product of many tokens,
tokens sorted by group and back, low-rank adapters of many requests.

Each function has the name of the C entry point it calls and only marshals
arguments, like the rest of the binding; shapes, strides, types and devices are
checked here, because the tensors carry what the C interface takes as sizes.
These calls are short on the GPU (a few microseconds for a decoding step), so
the checks are written to cost little: one test per tensor on the way, the
reason only for what fails it.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from . import BF16, F16, F32, SpmvError

_I32, _F32 = torch.int32, torch.float32
_HALF = (torch.float16, torch.uint16, torch.int16)      # fp16 data, or its raw bits
_WORD = (torch.uint32, torch.int32)                     # packed code words
_BYTE = (torch.int8, torch.uint8)
_CODE = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
_FUNCS = {}
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _func(name):
    f = _FUNCS.get(name)
    if f is None:
        f = _FUNCS[name] = getattr(_lib.load(), name)
    return f


def _check(status, name):
    if status != 0:
        raise SpmvError(status, name, _lib.load().spmv_last_error().decode(errors="replace"))


def _size(name, kind, *args):
    out = kind()
    _check(_func(name)(*[int(a) for a in args], ctypes.byref(out)), name)
    return out.value


def _launch(device, stream, name, *args):
    """The call on `stream` (None: the device's current one) with `device`
    current, since kernels and streams belong to a device."""
    index = device.index
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _current_device() == index:
        status = (_FUNCS.get(name) or _func(name))(*args, stream)
    else:
        with torch.cuda.device(device):
            status = _func(name)(*args, stream)
    if status != 0:
        _check(status, name)


def _stream_scope(stream, device):
    """The context whose current stream is `stream` (None: as it is)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream)


def _device(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.device


def _ptr(t, dtype, name, n, device):
    """Device pointer of a contiguous tensor of at least n elements on `device`."""
    try:
        if (t.dtype is dtype or t.dtype in dtype) and t.device == device and t.numel() >= n and t.is_contiguous():
            return t.data_ptr()
    except (AttributeError, TypeError):
        pass
    if t is None:
        raise ValueError(f"{name} is required")
    _device(t, name)
    if t.dtype is not dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    raise ValueError(f"{name} needs {n} elements, got {t.numel()}")


def _opt(t, dtype, name, n, device):
    return None if t is None else _ptr(t, dtype, name, n, device)


def _rows(t, dtype, name, n, width, device):
    """(device pointer, row stride) of an [n, width] tensor whose rows are contiguous."""
    try:
        if t.dtype is dtype or t.dtype in dtype:
            r, c = t.shape
            if r == n and c == width and t.device == device:
                ld, one = t.stride()
                if (one == 1 or c <= 1) and ld >= c and r > 1:
                    return t.data_ptr(), ld
                if r <= 1 and (one == 1 or c <= 1):
                    return t.data_ptr(), c
    except (AttributeError, TypeError, ValueError):
        pass
    _device(t, name)
    if t.dtype is not dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or tuple(t.shape) != (n, width):
        raise ValueError(f"{name} must have shape ({n}, {width}), got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    raise ValueError(f"the rows of {name} must be contiguous and must not overlap")


def _matrix(t, name):
    """(device, rows, width, device pointer, row stride) of a 2-D CUDA tensor
    whose rows are contiguous."""
    d = _device(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    n, width = t.shape
    ld, one = t.stride()
    if n > 1 and ld < width or one != 1 and width > 1:
        raise ValueError(f"the rows of {name} must be contiguous and must not overlap")
    return d, n, width, t.data_ptr(), ld if n > 1 else width


def _code(t, name):
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {t.dtype}")
    return code


def _ws(workspace, device):
    """(pointer, bytes) of a workspace tensor (None: NULL, 0)."""
    if workspace is None:
        return None, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
# MACKO for many tokens
# ---------------------------------------------------------------------------
def macko_spmm_plan_size(n_rows, n_cols) -> int:
    return _size("macko_spmm_plan_size", ctypes.c_size_t, n_rows, n_cols)


def macko_spmm_plan(n_rows, n_cols, mrow_ptr, codes, plan, stream=None, bdelta=4):
    """Fills `plan` (a uint8 CUDA tensor of macko_spmm_plan_size bytes) for
    the n_rows rows of all groups together."""
    d = _device(mrow_ptr, "mrow_ptr")
    pp, pb = _ws(plan, d)
    _launch(d, stream, "macko_spmm_plan", int(n_rows), int(n_cols), int(bdelta),
            _ptr(mrow_ptr, _I32, "mrow_ptr", n_rows + 1, d), _ptr(codes, _WORD, "codes", 0, d), pp, pb)
    return plan


def macko_spmm_workspace_size(n_groups, n_rows, n_cols, n_tok) -> int:
    return _size("macko_spmm_workspace_size", ctypes.c_size_t, n_groups, n_rows, n_cols, n_tok)


def _spmm(name, n_rows, n_cols, bdelta, mrow_ptr, codes, vals, plan, alpha, x, beta, y, workspace, tok_offsets, stream):
    d, n, width, xp, ldx = _matrix(x, "x")
    if width != n_cols or x.dtype not in _HALF:
        _rows(x, _HALF, "x", n, n_cols, d)                    # says which
    n_groups = 1 if tok_offsets is None else tok_offsets.numel() - 1
    yp, ldy = _rows(y, (torch.float16, _F32), "y", n, n_rows, d)
    pp, pb = _ws(plan, d)
    if pb < 4 * n_groups * n_rows * ((n_cols + 255) // 256 + 1):
        raise ValueError("plan is smaller than macko_spmm_plan_size")
    wp, wb = _ws(workspace, d)
    _launch(d, stream, name, n_groups, n_rows, n_cols, bdelta, _ptr(mrow_ptr, _I32, "mrow_ptr", n_groups * n_rows + 1, d),
            _ptr(codes, _WORD, "codes", 0, d), *vals(d, n_groups), pp, _opt(tok_offsets, _I32, "tok_offsets", 2, d), n,
            alpha, xp, ldx, beta, yp, _CODE[y.dtype], ldy, wp, wb)
    return y


def macko_spmm(n_rows, n_cols, mrow_ptr, codes, mvals, plan, alpha, x, beta, y, workspace=None, tok_offsets=None,
               stream=None, bdelta=4):
    """y = alpha * x W^T + beta * y for x [tokens, n_cols] fp16 and y [tokens,
    n_rows] fp32 or fp16; tok_offsets (int32 [groups + 1]): one stacked weight
    per group of tokens.  workspace: macko_spmm_workspace_size bytes, or those of
    a larger batch."""
    return _spmm("macko_spmm", int(n_rows), int(n_cols), int(bdelta), mrow_ptr, codes,
                 lambda d, g: (_ptr(mvals, _HALF, "mvals", 0, d),), plan, alpha, x, beta, y, workspace, tok_offsets, stream)


def macko_spmm_i8(n_rows, n_cols, mrow_ptr, codes, q, row_scale, plan, alpha, x, beta, y, workspace=None,
                  tok_offsets=None, stream=None, bdelta=4):
    return _spmm("macko_spmm_i8", int(n_rows), int(n_cols), int(bdelta), mrow_ptr, codes,
                 lambda d, g: (_ptr(q, _BYTE, "q", 0, d), _ptr(row_scale, _F32, "row_scale", g * n_rows, d)), plan, alpha,
                 x, beta, y, workspace, tok_offsets, stream)


class MackoMatrix:
    """One MACKO weight (or n_groups stacked ones) with its many-token plan.
    row_scale: the int8 values' scales, or None for fp16 values.  The plan is
    made on `stream`: other streams wait for it before they use the matrix, and
    it is kept until their calls are done."""

    def __init__(self, n_rows, n_cols, mrow_ptr, codes, vals, row_scale=None, n_groups=1, bdelta=4, stream=None):
        self.n_rows, self.n_cols, self.n_groups, self.bdelta = int(n_rows), int(n_cols), int(n_groups), int(bdelta)
        self.mrow_ptr, self.codes, self.vals, self.row_scale = mrow_ptr, codes, vals, row_scale
        if mrow_ptr.numel() != self.n_groups * self.n_rows + 1:
            raise ValueError(f"mrow_ptr must have {self.n_groups * self.n_rows + 1} elements")
        with _stream_scope(stream, mrow_ptr.device):
            self.plan = torch.empty(max(macko_spmm_plan_size(self.n_groups * self.n_rows, n_cols), 4), dtype=torch.uint8,
                                    device=mrow_ptr.device)
        macko_spmm_plan(self.n_groups * self.n_rows, n_cols, mrow_ptr, codes, self.plan, stream, bdelta)

    def workspace(self, n_tok):
        """A workspace for calls of n_tok tokens."""
        return torch.empty(macko_spmm_workspace_size(self.n_groups, self.n_rows, self.n_cols, n_tok), dtype=torch.uint8,
                           device=self.plan.device)

    def apply(self, x, y, alpha=1.0, beta=0.0, tok_offsets=None, workspace=None, stream=None):
        """y = alpha * x W^T + beta * y.  Without a workspace one is allocated
        for the call, in the order of the stream it runs on."""
        if (self.n_groups > 1 or tok_offsets is not None) and (
                tok_offsets is None or tok_offsets.numel() != self.n_groups + 1):
            raise ValueError(f"tok_offsets must have {self.n_groups + 1} elements")
        if workspace is None and x.dim() == 2:
            with _stream_scope(stream, self.plan.device):
                workspace = self.workspace(x.shape[0])
        if self.row_scale is None:
            return macko_spmm(self.n_rows, self.n_cols, self.mrow_ptr, self.codes, self.vals, self.plan, alpha, x, beta,
                              y, workspace, tok_offsets, stream, self.bdelta)
        return macko_spmm_i8(self.n_rows, self.n_cols, self.mrow_ptr, self.codes, self.vals, self.row_scale, self.plan,
                             alpha, x, beta, y, workspace, tok_offsets, stream, self.bdelta)


# ---------------------------------------------------------------------------
# Tokens sorted by group and back
# ---------------------------------------------------------------------------
def route_tile_count(n_slots, n_groups) -> int:
    return _size("route_tile_count", ctypes.c_int32, n_slots, n_groups)


def route_workspace_size(n_slots, n_groups) -> int:
    return _size("route_workspace_size", ctypes.c_size_t, n_slots, n_groups)


def route_plan(n_groups, keys, offsets, order, pos, tiles, workspace=None, stream=None):
    """Fills offsets [n_groups + 1], order and pos [slots] and tiles
    [route_tile_count, 4] (int32 CUDA tensors) from keys (int32, any shape)."""
    d, n = _device(keys, "keys"), keys.numel()
    n_tiles = (n + 15 * min(n_groups + 1, n)) // 16
    wp, wb = _ws(workspace, d)
    _launch(d, stream, "route_plan", n, n_groups, _ptr(keys, _I32, "keys", n, d),
            _ptr(offsets, _I32, "offsets", n_groups + 1, d), _ptr(order, _I32, "order", n, d), _ptr(pos, _I32, "pos", n, d),
            _ptr(tiles, _I32, "tiles", 4 * n_tiles, d), wp, wb)


def _top_k(pos, n_tok):
    if pos.dim() != 2 or pos.shape[0] != n_tok or pos.shape[1] < 1:
        raise ValueError(f"pos must have shape ({n_tok}, top_k), got {tuple(pos.shape)}")
    return pos.shape[1]


def route_gather(x, pos, xs, weights=None, stream=None):
    """xs[pos[t, c]] = weights[t, c] * x[t]; pos: [tokens, top_k]."""
    k = _top_k(pos, x.shape[0])
    d, n, dim, xp, ldx = _matrix(x, "x")
    sp, lds = _rows(xs, x.dtype, "xs", n * k, dim, d)
    _launch(d, stream, "route_gather", n, k, dim, _code(x, "x"), _ptr(pos, _I32, "pos", n * k, d),
            _opt(weights, _F32, "weights", n * k, d), xp, ldx, sp, lds)
    return xs


def route_combine(ys, pos, y, weights=None, stream=None):
    """y[t] = sum_c weights[t, c] * ys[pos[t, c]]; pos: [tokens, top_k]."""
    k = _top_k(pos, y.shape[0])
    d, n, dim, yp, ldy = _matrix(y, "y")
    sp, lds = _rows(ys, y.dtype, "ys", n * k, dim, d)
    _launch(d, stream, "route_combine", n, k, dim, _code(y, "y"), _ptr(pos, _I32, "pos", n * k, d),
            _opt(weights, _F32, "weights", n * k, d), sp, lds, yp, ldy)
    return y


def route_combine_grad(dy, ys, pos, weights, dys, dw, stream=None):
    """dys[pos[t, c]] = weights[t, c] * dy[t]; dw[t, c] = <ys[pos[t, c]], dy[t]>."""
    k = _top_k(pos, dy.shape[0])
    d, n, dim, gp, ldg = _matrix(dy, "dy")
    sp, lds = _rows(ys, dy.dtype, "ys", n * k, dim, d)
    op, ldo = _rows(dys, dy.dtype, "dys", n * k, dim, d)
    _launch(d, stream, "route_combine_grad", n, k, dim, _code(dy, "dy"), gp, ldg, sp, lds, _ptr(pos, _I32, "pos", n * k, d),
            _opt(weights, _F32, "weights", n * k, d), op, ldo, _ptr(dw, _F32, "dw", n * k, d))
    return dys, dw


class RoutePlan:
    """The plan of a batch of n_tok tokens with top_k choices of n_groups
    groups each: build() sorts, gather() and combine() move rows there and
    back.  One plan serves every layer that shares the batch's keys.  Its arrays
    are allocated on the current stream: another one that build() is to run on
    waits for it first."""

    def __init__(self, n_tok, top_k, n_groups, device="cuda"):
        self.n_tok, self.top_k, self.n_groups = int(n_tok), int(top_k), int(n_groups)
        n = self.n_tok * self.top_k
        new = lambda *shape: torch.empty(*shape, dtype=torch.int32, device=device)  # noqa: E731
        self.offsets, self.order, self.pos = new(self.n_groups + 1), new(n), new(self.n_tok, self.top_k)
        self.tiles = new(route_tile_count(n, n_groups), 4)
        self.workspace = torch.empty(route_workspace_size(n, n_groups), dtype=torch.uint8, device=device)

    def build(self, keys, stream=None):
        """keys: int32 [n_tok, top_k] (or flat); outside [0, n_groups): dropped."""
        if keys.numel() != self.n_tok * self.top_k:
            raise ValueError(f"keys must have {self.n_tok * self.top_k} elements, got {keys.numel()}")
        route_plan(self.n_groups, keys, self.offsets, self.order, self.pos, self.tiles, self.workspace, stream)
        return self

    def gather(self, x, xs, weights=None, stream=None):
        return route_gather(x, self.pos, xs, weights, stream)

    def combine(self, ys, y, weights=None, stream=None):
        return route_combine(ys, self.pos, y, weights, stream)

    def combine_grad(self, dy, ys, weights, dys, dw, stream=None):
        return route_combine_grad(dy, ys, self.pos, weights, dys, dw, stream)


# ---------------------------------------------------------------------------
# Low-rank adapters of many requests
# ---------------------------------------------------------------------------
def lora_workspace_size(n_tok, max_rank) -> int:
    return _size("lora_workspace_size", ctypes.c_size_t, n_tok, max_rank)


def _lora_args(ranks, scale, A, B, order, offsets, tiles, x):
    d, n, n_in, xp, ldx = _matrix(x, "x")
    dt = x.dtype
    if dt is not torch.float16 and dt is not torch.bfloat16:
        raise TypeError(f"x must be float16 or bfloat16, got {dt}")
    if A.dim() != 3 or B.dim() != 3 or A.shape[:2] != B.shape[:2]:
        raise ValueError(f"A and B must be [adapters, rank, width], got {tuple(A.shape)} and {tuple(B.shape)}")
    n_ad, r, width = A.shape
    n_out = B.shape[2]
    if width != n_in:
        raise ValueError(f"x must have {width} columns like A, got {n_in}")
    if offsets.numel() != n_ad + 1 or order.numel() != n:
        raise ValueError("the plan is not one of x's tokens and A's adapters")
    return d, (n, n_in, n_out, n_ad, r, _opt(ranks, _I32, "ranks", n_ad, d), _opt(scale, _F32, "scale", n_ad, d),
               _ptr(A, dt, "A", 0, d), _ptr(B, dt, "B", 0, d), _CODE[dt], _ptr(order, _I32, "order", n, d),
               _ptr(offsets, _I32, "offsets", n_ad + 1, d), _ptr(tiles, _I32, "tiles", 0, d), tiles.numel() // 4, xp, ldx)


def lora_apply(ranks, scale, A, B, order, offsets, tiles, x, y_in, y, workspace, stream=None):
    """y[t] = y_in[t] + scale[a] * B[a]^T (A[a] x[t]) for token t's adapter a
    (y_in: None for zeros, or y itself).  A [adapters, rank, n_in] and
    B [adapters, rank, n_out]; order, offsets, tiles: a RoutePlan's, of one
    choice per token.  The gradient in x: A and B exchanged, dy for x."""
    d, a = _lora_args(ranks, scale, A, B, order, offsets, tiles, x)
    yp, ldy = _rows(y, (x.dtype, _F32), "y", a[0], a[2], d)
    ip, ldi = (None, 0) if y_in is None else (yp, ldy) if y_in is y else _rows(y_in, y.dtype, "y_in", a[0], a[2], d)
    wp, wb = _ws(workspace, d)
    _launch(d, stream, "lora_apply", *a, ip, ldi, yp, _CODE[y.dtype], ldy, wp, wb)
    return y


def lora_grad(ranks, scale, A, B, order, offsets, tiles, x, dy, dA, dB, workspace, stream=None):
    """Weight gradients of lora_apply, fp32: dA like A, dB like B."""
    d, a = _lora_args(ranks, scale, A, B, order, offsets, tiles, x)
    if dA.shape != A.shape or dB.shape != B.shape:
        raise ValueError("dA and dB must have the shapes of A and B")
    gp, ldg = _rows(dy, x.dtype, "dy", a[0], a[2], d)
    wp, wb = _ws(workspace, d)
    _launch(d, stream, "lora_grad", *a, gp, ldg, _ptr(dA, _F32, "dA", 0, d), _ptr(dB, _F32, "dB", 0, d), wp, wb)
    return dA, dB
