"""Plain references in 64 bits of the 4-bit products, the expert layer and the
embeddings, and their error bounds (counted as in op_refs)."""
from __future__ import annotations

import numpy as np
import torch

from op_refs import ADD, f64, rounded

PLACE = [(e >> 1) + 4 * (e & 1) for e in range(8)]


def blocks(n_cols):
    return (n_cols + 127) // 128


def pack(q):
    """int32 words [rows, 16 * blocks] of codes q [rows, 128 * blocks]."""
    q = np.asarray(q, dtype=np.uint32)
    n, width = q.shape
    words = np.zeros((n, width // 8), np.uint32)
    for b in range(width // 128):
        for j in range(4):
            for m in range(4):
                for e in range(8):
                    words[:, 16 * b + 4 * j + m] |= q[:, 128 * b + 32 * m + 8 * j + e] << np.uint32(4 * PLACE[e])
    return torch.from_numpy(words.view(np.int32))


def unpack(words):
    w = words.cpu().numpy().view(np.uint32)
    n = w.shape[0]
    q = np.zeros((n, w.shape[1] * 8), np.int64)
    for b in range(w.shape[1] // 16):
        for j in range(4):
            for m in range(4):
                for e in range(8):
                    q[:, 128 * b + 32 * m + 8 * j + e] = (w[:, 16 * b + 4 * j + m] >> np.uint32(4 * PLACE[e])) & 15
    return q


def dense(words, scales, zeros, group, n_cols):
    """The weight in float64 [rows, n_cols]."""
    q = torch.from_numpy(unpack(words)).double()
    z = torch.full(scales.shape, 8.0, dtype=torch.float64) if zeros is None else (zeros.cpu() & 15).double()
    w = (q - torch.repeat_interleave(z, group, 1)) * torch.repeat_interleave(f64(scales), group, 1)
    return w[:, :n_cols]


def weight(rows, cols, group, dtype, zeros, seed, scale=None):
    """(codes, scales, zeros) on the CPU, codes over the whole range, the filled-up columns as well."""
    g = torch.Generator().manual_seed(seed)
    n = blocks(cols) * 128
    q = torch.randint(0, 16, (rows, n), generator=g)
    s = (torch.rand(rows, n // group, generator=g) + 0.25) * (0.05 if scale is None else scale)
    z = torch.randint(0, 16, s.shape, generator=g).to(torch.uint8) if zeros else None
    return pack(q.numpy()), s.to(dtype), z


def product_steps(n_cols, group):
    """fp32 additions that a product passes through: in the matrix cores up to 36 for a
    group, then one per group, 16 waves' sums, 32 parts of the columns, scale and alpha."""
    return 36 + blocks(n_cols) * (128 // group) + 16 + 32 + 8


def matmul(w, x, alpha, beta, y_in, y_dtype, group):
    x = f64(x)
    ref = alpha * (x @ w.t())
    mag = abs(alpha) * (x.abs() @ w.abs().t())
    bound = mag * (product_steps(x.shape[1], group) * ADD)
    if beta != 0.0:
        ref = ref + beta * f64(y_in)
        bound = bound + (abs(beta) * f64(y_in).abs() + mag) * 2 * ADD
    return ref, bound + rounded(ref.abs() + bound, y_dtype)


def moe(keys, weights, up, down, x, y_dtype, group):
    """(y, bound): up [experts, 2 inter, dim], down [experts, dim, inter] in float64."""
    x = f64(x)
    T, dim = x.shape
    inter = down.shape[2]
    y = torch.zeros(T, dim, dtype=torch.float64)
    bound = torch.zeros_like(y)
    mag = torch.zeros_like(y)
    c1 = product_steps(dim, group) * ADD
    c2 = (3 * product_steps(inter, group) + keys.shape[1] + 8) * ADD
    for t in range(T):
        for c in range(keys.shape[1]):
            e = int(keys[t, c])
            if not 0 <= e < up.shape[0]:
                continue
            gu = up[e] @ x[t]
            d = (up[e].abs() @ x[t].abs()) * c1
            g, u, dg, du = gu[:inter], gu[inter:], d[:inter], d[inter:]
            sig = torch.sigmoid(g)
            h = g * sig * u
            # |silu'| < 1.1; silu and the product round a few times; three bf16 numbers cut at 24 bits
            dh = 1.1 * dg * (u.abs() + du) + (g * sig).abs() * du + h.abs() * 12 * 2.0 ** -24
            w = 1.0 if weights is None else float(weights[t, c])
            y[t] += w * (down[e] @ h)
            m = down[e].abs() @ (h.abs() + dh)
            bound[t] += abs(w) * (down[e].abs() @ dh)
            mag[t] += abs(w) * m
    bound = bound + mag * c2
    return y, bound + rounded(y.abs() + bound, y_dtype)


def embed(ids, table, scale, y_dtype):
    ids = np.asarray(ids)
    ok = torch.from_numpy((ids >= 0) & (ids < table.shape[0]))
    t = f64(table)
    y = torch.zeros(len(ids), t.shape[1], dtype=torch.float64)
    y[ok] = scale * t[torch.from_numpy(ids.astype(np.int64))[ok]]
    return y, y.abs() * 2.0 ** -24 + rounded(y, y_dtype)


def embed_grad(ids, dy, n_vocab, scale, first=None):
    """(dtable, bound); fp32 additions: one per token of a row, whatever their grouping."""
    ids, dy = np.asarray(ids).astype(np.int64), f64(dy)
    ok = torch.from_numpy((ids >= 0) & (ids < n_vocab))
    at = torch.from_numpy(ids)[ok]
    out = torch.zeros(n_vocab, dy.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    out.index_add_(0, at, dy[ok])
    mag.index_add_(0, at, dy[ok].abs())
    n = torch.bincount(at, minlength=n_vocab).double()[:, None]
    out, bound = scale * out, abs(scale) * mag * (n + 2) * 2.0 ** -24 + 2.0 ** -149
    if first is not None:
        out = out + f64(first)
        bound = bound + (f64(first).abs() + abs(scale) * mag) * 2.0 ** -23
    bound[(n == 0)[:, 0]] = 0.0
    return out, bound
