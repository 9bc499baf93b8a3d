"""Dense weights of 4 bits (products, expert layers) and token embeddings of the
binding.

Each function has the name of the C entry point it calls and only marshals
arguments; shapes, strides, types and devices are checked here, as for the other
operators of many tokens.
"""
from __future__ import annotations

import ctypes

import torch

from .tokens import (_CODE, _F32, _I32, _WORD, _code, _device, _launch, _matrix, _opt, _ptr, _rows, _size,
                     _stream_scope, _ws)

_HALF_TYPES = (torch.float16, torch.bfloat16)


def _groups(n_cols, group):
    """Groups of a row, its last block of 128 columns filled up."""
    return (n_cols + 127) // 128 * (128 // group)


def _tensor(t, name):
    """Before a tensor's shape or type is asked for: the rest is checked with its pointer."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")


def _group(group):
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    return group


# ---------------------------------------------------------------------------
# Weights of 4 bits
# ---------------------------------------------------------------------------
def q4_quantize(w, codes, scales, zeros=None, group=128, stream=None):
    """Fills codes (int32 [rows, 16 * blocks]), scales (float16 or bfloat16 [rows,
    groups]) and, if given, zeros (uint8 [rows, groups]) from w [rows, cols]; a row
    has ceil(cols / 128) blocks of 128 / group groups."""
    d, n, width, wp, ldw = _matrix(w, "w")
    blocks, per = (width + 127) // 128, _groups(width, _group(group))
    _tensor(scales, "scales")
    if scales.dtype not in _HALF_TYPES:
        raise TypeError(f"scales must be float16 or bfloat16, got {scales.dtype}")
    _launch(d, stream, "q4_quantize", n, width, group, wp, _code(w, "w"), ldw, _CODE[scales.dtype],
            _ptr(codes, _WORD, "codes", n * blocks * 16, d), _ptr(scales, scales.dtype, "scales", n * per, d),
            _opt(zeros, torch.uint8, "zeros", n * per, d))
    return codes, scales, zeros


def q4_tiles_size(n_rows, n_cols, group=128, with_zeros=False) -> int:
    return _size("q4_tiles_size", ctypes.c_size_t, n_rows, n_cols, group, with_zeros)


def q4_tiles(n_rows, n_cols, codes, scales, zeros, tiles, group=128, stream=None):
    """Fills tiles (uint8, q4_tiles_size bytes), what the products read, from the
    rows' codes, scales and zero points (or None)."""
    n_rows, n_cols = int(n_rows), int(n_cols)
    d, per = _device(codes, "codes"), n_rows * _groups(n_cols, _group(group))
    if not isinstance(scales, torch.Tensor) or scales.dtype not in _HALF_TYPES:
        raise TypeError("scales must be a float16 or bfloat16 tensor")
    tp, tb = _ws(tiles, d)
    _launch(d, stream, "q4_tiles", n_rows, n_cols, group,
            _ptr(codes, _WORD, "codes", n_rows * ((n_cols + 127) // 128) * 16, d),
            _ptr(scales, scales.dtype, "scales", per, d), _opt(zeros, torch.uint8, "zeros", per, d), tp, tb)
    return tiles


def q4_workspace_size(n_rows, n_cols, n_tok) -> int:
    return _size("q4_workspace_size", ctypes.c_size_t, n_rows, n_cols, n_tok)


def q4_matmul(n_rows, n_cols, tiles, alpha, x, beta, y, workspace=None, group=128, with_zeros=False, stream=None):
    """y = alpha * x W^T + beta * y for x [tokens, n_cols] of the scales' type and y
    [tokens, n_rows] of the same type or fp32.  workspace: q4_workspace_size bytes for
    these tokens or more."""
    d, n, width, xp, ldx = _matrix(x, "x")
    dt = x.dtype
    if dt not in _HALF_TYPES:
        raise TypeError(f"x must be float16 or bfloat16, got {dt}")
    if width != n_cols:
        raise ValueError(f"x must have {n_cols} columns, got {width}")
    yp, ldy = _rows(y, (dt, _F32), "y", n, n_rows, d)
    wp, wb = _ws(workspace, d)
    tp, tb = _ws(tiles, d)
    if tb < (n_rows + 15) // 16 * ((n_cols + 127) // 128) * (1024 + 128 // _group(group) * (48 if with_zeros else 32)):
        raise ValueError("tiles are smaller than q4_tiles_size")
    _launch(d, stream, "q4_matmul", n_rows, n_cols, group, with_zeros, tp, _CODE[dt], n, alpha, xp, ldx, beta, yp,
            _CODE[y.dtype], ldy, wp, wb)
    return y


class Q4Matrix:
    """One 4-bit weight, or n_groups stacked ones (the experts of moe_apply), arranged
    for the products from codes, scales and zero points (or None) in the layout of
    include/spmv.h, which may be freed afterwards.  It is made on `stream`: before
    another stream uses the matrix the caller makes it wait, and keeps the matrix until
    the calls there are done."""

    def __init__(self, n_rows, n_cols, codes, scales, zeros=None, group=128, n_groups=1, stream=None):
        self.n_rows, self.n_cols, self.n_groups, self.group = int(n_rows), int(n_cols), int(n_groups), _group(group)
        self.with_zeros = int(zeros is not None)
        d, total = _device(codes, "codes"), self.n_rows * self.n_groups
        if total > 0x7fffffff:
            raise ValueError(f"{total} rows in all do not fit int32")
        with _stream_scope(stream, d):
            self.tiles = torch.empty(q4_tiles_size(total, n_cols, group, self.with_zeros), dtype=torch.uint8, device=d)
        q4_tiles(total, n_cols, codes, scales, zeros, self.tiles, group, stream)
        self.dtype = scales.dtype

    @classmethod
    def quantize(cls, w, group=128, dtype=None, zeros=False, stream=None):
        """The weight w [rows, cols], or [n_groups, rows, cols], in 4 bits, with zero
        points if `zeros`; dtype: the scales' type (w's, or float16 for fp32)."""
        d = _device(w, "w")
        if w.dim() not in (2, 3):
            raise ValueError(f"w must be 2-D or 3-D, got shape {tuple(w.shape)}")
        n_groups, (rows, cols) = w.shape[0] if w.dim() == 3 else 1, w.shape[-2:]
        dtype = dtype or (w.dtype if w.dtype in _HALF_TYPES else torch.float16)
        shape = (n_groups * rows, _groups(cols, _group(group)))
        with _stream_scope(stream, d):
            w = w.reshape(n_groups * rows, cols) if w.dim() == 3 else w      # a copy if strided, in the stream's order
            codes = torch.empty(w.shape[0], (cols + 127) // 128 * 16, dtype=_I32, device=w.device)
            scales = torch.empty(shape, dtype=dtype, device=w.device)
            zp = torch.empty(shape, dtype=torch.uint8, device=w.device) if zeros else None
        q4_quantize(w, codes, scales, zp, group, stream)
        return cls(rows, cols, codes, scales, zp, group, n_groups, stream)

    def workspace(self, n_tok):
        """A workspace for calls of up to n_tok tokens."""
        return torch.empty(q4_workspace_size(self.n_rows, self.n_cols, n_tok), dtype=torch.uint8,
                           device=self.tiles.device)

    def apply(self, x, y, alpha=1.0, beta=0.0, workspace=None, stream=None):
        """y = alpha * x W^T + beta * y (of a single weight).  Without a workspace one
        is allocated for the call, in the order of the stream it runs on."""
        if self.n_groups != 1:
            raise ValueError("apply takes a single weight; stacked ones are moe_apply's")
        d, n, width, xp, ldx = _matrix(x, "x")
        dt = x.dtype
        if dt is not self.dtype:
            raise TypeError(f"x must be {self.dtype} like the scales, got {dt}")
        if width != self.n_cols:
            raise ValueError(f"x must have {self.n_cols} columns, got {width}")
        if d != self.tiles.device:
            raise ValueError(f"x is on {d}, not on {self.tiles.device}")
        if workspace is None:
            with _stream_scope(stream, d):
                workspace = self.workspace(n)
        yp, ldy = _rows(y, (dt, _F32), "y", n, self.n_rows, d)
        wp, wb = _ws(workspace, d)
        _launch(d, stream, "q4_matmul", self.n_rows, width, self.group, self.with_zeros, self.tiles.data_ptr(), _CODE[dt],
                n, alpha, xp, ldx, beta, yp, _CODE[y.dtype], ldy, wp, wb)
        return y


# ---------------------------------------------------------------------------
# A layer of experts for a few tokens
# ---------------------------------------------------------------------------
def moe_workspace_size(n_tok, top_k, dim, inter) -> int:
    return _size("moe_workspace_size", ctypes.c_size_t, n_tok, top_k, dim, inter)


def moe_apply(keys, weights, gate_up, down, x, y, workspace, stream=None):
    """y[t] = sum_c weights[t, c] * down_e(silu(gate_e x[t]) * (up_e x[t])), e = keys[t, c].
    keys: int32 [tokens, top_k]; weights: fp32 of the same shape, or None for ones;
    gate_up: a Q4Matrix of n_groups experts with the gate's rows before the up's
    (2 inter x dim), down: one of dim x inter.  At most 256 tokens."""
    d, n, dim, xp, ldx = _matrix(x, "x")
    dt = x.dtype
    _tensor(keys, "keys")
    if keys.dim() != 2 or keys.shape[0] != n or keys.shape[1] < 1:
        raise ValueError(f"keys must have shape ({n}, top_k), got {tuple(keys.shape)}")
    if weights is not None:
        _tensor(weights, "weights")
        if weights.shape != keys.shape:
            raise ValueError(f"weights must have the shape of keys, got {tuple(weights.shape)}")
    if not isinstance(gate_up, Q4Matrix) or not isinstance(down, Q4Matrix):
        raise TypeError("gate_up and down must be Q4Matrix")
    k, e, inter = keys.shape[1], gate_up.n_groups, down.n_cols
    if gate_up.n_cols != dim or gate_up.n_rows != 2 * inter or down.n_rows != dim or down.n_groups != e:
        raise ValueError(f"{e} x {gate_up.n_rows} x {gate_up.n_cols} and {down.n_groups} x {down.n_rows} x {down.n_cols} "
                         f"are not the weights of a layer of width {dim}")
    if gate_up.group != down.group or gate_up.with_zeros != down.with_zeros:
        raise ValueError("the two weights must have the same group size, and both zero points or neither")
    if gate_up.dtype is not dt or down.dtype is not dt:
        raise TypeError(f"x must be of the scales' type, got {dt}, {gate_up.dtype} and {down.dtype}")
    yp, ldy = _rows(y, (dt, _F32), "y", n, dim, d)
    wp, wb = _ws(workspace, d)
    (up, _), (dn, _) = _ws(gate_up.tiles, d), _ws(down.tiles, d)
    _launch(d, stream, "moe_apply", n, k, e, dim, inter, down.group, down.with_zeros, _ptr(keys, _I32, "keys", n * k, d),
            _opt(weights, _F32, "weights", n * k, d), up, dn, _CODE[dt], xp, ldx, yp, _CODE[y.dtype], ldy, wp, wb)
    return y


# ---------------------------------------------------------------------------
# Token embeddings
# ---------------------------------------------------------------------------
def embed_lookup(ids, table, y, scale=1.0, stream=None):
    """y[t] = scale * table[ids[t]], zeros for ids outside the table.  ids: int32
    [tokens]; y [tokens, dim] of the table's type or fp32."""
    d, v, dim, tp, ldt = _matrix(table, "table")
    _tensor(ids, "ids")
    n = ids.numel()
    yp, ldy = _rows(y, (table.dtype, _F32), "y", n, dim, d)
    _launch(d, stream, "embed_lookup", n, v, dim, _code(table, "table"), _ptr(ids, _I32, "ids", n, d), tp, ldt, scale, yp,
            _CODE[y.dtype], ldy)
    return y


def embed_grad_workspace_size(n_tok, n_vocab, dim) -> int:
    return _size("embed_grad_workspace_size", ctypes.c_size_t, n_tok, n_vocab, dim)


def embed_grad(ids, dy, dtable, workspace, scale=1.0, accumulate=False, stream=None):
    """dtable[v] = scale * sum of dy[t] over ids[t] = v (fp32 [vocabulary, dim]), or
    added to it with `accumulate`."""
    d, n, dim, gp, ldg = _matrix(dy, "dy")
    _tensor(ids, "ids")
    _tensor(dtable, "dtable")
    if ids.numel() != n:
        raise ValueError(f"ids must have {n} elements, got {ids.numel()}")
    if dtable.dim() != 2:
        raise ValueError(f"dtable must be 2-D, got shape {tuple(dtable.shape)}")
    v = dtable.shape[0]
    tp, ldt = _rows(dtable, _F32, "dtable", v, dim, d)
    wp, wb = _ws(workspace, d)
    _launch(d, stream, "embed_grad", n, v, dim, _code(dy, "dy"), _ptr(ids, _I32, "ids", n, d), gp, ldg, scale,
            int(accumulate), tp, ldt, wp, wb)
    return dtable
