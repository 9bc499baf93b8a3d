"""Plain references in 64 bits of the many-token operators, and their error
bounds.  EPS2 is half a step of a type relative to a value (the error of one
rounding); TINY the largest rounding error next to zero."""
from __future__ import annotations

import numpy as np
import torch

EPS2 = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
# fp32 sums are counted as one step of 2^-23 per addition: half a step for
# round to nearest, a whole one where the matrix cores truncate.
ADD = 2.0 ** -23


def f64(t):
    return t.detach().to("cpu").double()


def check(got, ref, bound, what=""):
    """Element by element: |got - ref| <= bound (float64 CPU tensors)."""
    g = f64(got)
    assert g.shape == ref.shape, f"{what}: shape {tuple(g.shape)} is not {tuple(ref.shape)}"
    bad = ~((g - ref).abs() <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at {i}: "
                             f"got {float(g[i])!r} ref {float(ref[i])!r} bound {float(bound[i])!r}")


def rounded(ref, dtype):
    """Bound of rounding a value near ref to dtype."""
    return ref.abs() * EPS2[dtype] * (1 + EPS2[dtype]) + TINY[dtype]


# ---------------------------------------------------------------------------
def route_plan(keys, n_groups):
    k = np.asarray(keys, dtype=np.int64).reshape(-1)
    ok = (k >= 0) & (k < n_groups)
    kk = np.where(ok, k, n_groups)
    order = np.argsort(kk, kind="stable")
    pos = np.empty(len(k), np.int64)
    pos[order] = np.arange(len(k))
    pos[~ok] = -1
    counts = np.bincount(kk, minlength=n_groups + 1)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    tiles = []
    for g in range(n_groups + 1):
        for b in range(offsets[g], offsets[g + 1], 16):
            tiles.append((g if g < n_groups else -1, b, min(b + 16, offsets[g + 1]), offsets[g]))
    return offsets[:n_groups + 1], order, pos, tiles


# ---------------------------------------------------------------------------
def lora(keys, ranks, scale, A, B, x, y_in, n_terms_bits, y_dtype):
    """(y, bound): ranks, scale as Python lists.  n_terms_bits: bits of the
    rank vector as an operand (fp16 pairs 22, bf16 pairs 16, triples 24)."""
    x, A, B = f64(x), f64(A), f64(B)
    T, K = x.shape
    N = B.shape[2]
    y = torch.zeros(T, N, dtype=torch.float64) if y_in is None else f64(y_in).clone()
    bound = torch.zeros(T, N, dtype=torch.float64)
    for t in range(T):
        a = int(keys[t])
        if not 0 <= a < A.shape[0] or ranks[a] <= 0:
            continue
        r = min(ranks[a], A.shape[1])
        h = A[a, :r] @ x[t]
        # K products added in fp32, in chains of at most K / 32 + 32 and 40 partial sums
        dh = (A[a, :r].abs() @ x[t].abs()) * ((K / 32 + 72) * ADD)
        dh = dh + h.abs() * 2.0 ** -n_terms_bits + h.abs().max() * 2.0 ** -25
        s = abs(scale[a])
        d = h @ B[a, :r]
        mag = (h.abs() + dh) @ B[a, :r].abs()
        y[t] = y[t] + scale[a] * d
        # three terms of r products each, then scale, product and sum
        bound[t] = s * (dh @ B[a, :r].abs() + mag * ((3 * r + 6) * ADD)) + (y[t].abs() + s * mag) * 2 * ADD
    same = (bound == 0).all(dim=1)
    total = bound + rounded(y.abs() + bound, y_dtype)
    total[same] = 0.0                      # rows without an adapter are copies
    return y, total


def lora_grad(keys, ranks, scale, A, B, x, dy):
    """(dA, bound, dB, bound)."""
    x, dy, A, B = f64(x), f64(dy), f64(A), f64(B)
    n, R = A.shape[:2]
    out = [torch.zeros_like(A), torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(B)]
    keys = np.asarray(keys)
    for a in range(n):
        r = max(0, min(ranks[a], R))
        at = torch.from_numpy(np.flatnonzero(keys == a))
        if r == 0 or len(at) == 0:
            continue
        for k, (W, u, v) in enumerate(((B, dy, x), (A, x, dy))):
            W, u, v = W[a, :r], u[at], v[at]
            g = u @ W.t()
            dg = (u.abs() @ W.abs().t()) * ((u.shape[1] / 32 + 72) * ADD)
            # two 16-bit terms: 22 bits; brought to the scale of the largest of 32
            # tokens, each term is rounded to a multiple of 2^-24 of it, or dropped below 2^-24
            dg = dg + g.abs() * 2.0 ** -22 + g.abs().max() * 2.0 ** -23
            s = abs(scale[a])
            out[2 * k][a, :r] = scale[a] * (g.t() @ v)
            mag = (g.abs() + dg).t() @ v.abs()
            out[2 * k + 1][a, :r] = s * (dg.t() @ v.abs() + mag * ((3 * 32 + len(at) / 32 + 16) * ADD))
    return out


# ---------------------------------------------------------------------------
def spmm(dense, x, alpha, beta, y_in, y_dtype):
    """(y, bound) of alpha * x dense^T + beta * y_in; dense: float64 [rows, cols]."""
    x = f64(x)
    K = x.shape[1]
    ref = alpha * (x @ dense.t())
    mag = abs(alpha) * (x.abs() @ dense.abs().t())
    bound = mag * ((K / 32 + 72 + 4) * ADD)
    if beta != 0.0:
        ref = ref + beta * f64(y_in)
        bound = bound + (abs(beta) * f64(y_in).abs() + mag) * 2 * ADD
    return ref, bound + rounded(ref.abs() + bound, y_dtype)
