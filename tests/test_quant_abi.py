"""CPU-side checks of the C entry points of 4-bit weights, expert layers and
embeddings (no kernel is launched): sizes, refusals with their statuses, calls
that have nothing to do, and what the binding refuses."""
import ctypes

import numpy as np
import pytest

import sparse_matrix_vector_amd as S

OK, VALUE, OVERFLOW, UNSUPPORTED = 0, 1, 4, 5
P = 4096                                     # a pointer that is aligned and never followed
F16, BF16, F32 = 0, 1, 2


def _quantize(rows=8, cols=100, group=32, w=P, wdt=F32, ldw=100, dt=F16, codes=P, scales=P, zeros=None):
    return S.lib().q4_quantize(rows, cols, group, w, wdt, ldw, dt, codes, scales, zeros, None)


def test_quantize_refusals():
    assert _quantize(rows=-1) == VALUE and _quantize(cols=-1) == VALUE
    for g in (0, 16, 33, 96, 256):
        assert _quantize(group=g) == VALUE, g
    assert _quantize(wdt=3) == VALUE and _quantize(dt=-1) == VALUE and _quantize(dt=F32) == UNSUPPORTED
    assert _quantize(ldw=99) == VALUE
    for k in ("w", "codes", "scales"):
        assert _quantize(**{k: None}) == VALUE, k
    assert _quantize(rows=2 ** 31 - 1, cols=2 ** 20, ldw=2 ** 20) == OVERFLOW
    assert _quantize(rows=0, w=None) == OK and _quantize(cols=0, ldw=0, w=None) == OK


def _tiles(rows=20, cols=300, group=64, codes=P, scales=P, zeros=None, tiles=P, tb=1 << 20):
    return S.lib().q4_tiles(rows, cols, group, codes, scales, zeros, tiles, tb, None)


def test_tiles_sizes_and_refusals():
    assert S.q4_tiles_size(20, 300, 64) == 2 * 3 * (1024 + 2 * 32)
    assert S.q4_tiles_size(16, 128, 32, True) == 1024 + 4 * 48 and S.q4_tiles_size(1, 1, 128) == 1056
    assert S.q4_tiles_size(0, 300) == 0 and S.q4_tiles_size(20, 0) == 0
    z = ctypes.c_size_t()
    L = S.lib()
    assert L.q4_tiles_size(-1, 4, 32, 0, ctypes.byref(z)) == VALUE and L.q4_tiles_size(4, -1, 32, 0, ctypes.byref(z)) == VALUE
    assert L.q4_tiles_size(4, 4, 31, 0, ctypes.byref(z)) == VALUE and L.q4_tiles_size(4, 4, 32, 0, None) == VALUE
    assert _tiles(rows=-1) == VALUE and _tiles(group=16) == VALUE
    for k in ("codes", "scales", "tiles"):
        assert _tiles(**{k: None}) == VALUE, k
    assert _tiles(tb=S.q4_tiles_size(20, 300, 64) - 1) == VALUE
    assert _tiles(zeros=P, tb=S.q4_tiles_size(20, 300, 64)) == VALUE
    assert _tiles(codes=P + 8) == UNSUPPORTED and _tiles(tiles=P + 8) == UNSUPPORTED
    assert _tiles(rows=2 ** 31 - 1, cols=2 ** 20, tb=2 ** 62) == OVERFLOW
    assert _tiles(rows=0, codes=None) == OK and _tiles(cols=0, tiles=None) == OK


def _matmul(rows=40, cols=100, group=64, zp=0, tiles=P, dt=F16, n=4, x=P, ldx=100, beta=0.0, y=P, ydt=F32, ldy=40, ws=None,
            wsb=0):
    return S.lib().q4_matmul(rows, cols, group, zp, tiles, dt, n, 1.0, x, ldx, beta, y, ydt, ldy, ws, wsb, None)


def test_matmul_refusals():
    assert _matmul(rows=-1) == VALUE and _matmul(cols=-1) == VALUE and _matmul(n=-1) == VALUE
    assert _matmul(group=48) == VALUE and _matmul(dt=5) == VALUE and _matmul(ydt=5) == VALUE
    assert _matmul(dt=F32) == UNSUPPORTED and _matmul(dt=F16, ydt=BF16) == UNSUPPORTED
    assert _matmul(ldx=99) == VALUE and _matmul(ldy=39) == VALUE
    assert _matmul(cols=2 ** 30 + 1, ldx=2 ** 31) == UNSUPPORTED
    assert _matmul(rows=2 ** 31 - 1, cols=4, ldx=4, ldy=2 ** 31) == OVERFLOW
    for k in ("tiles", "x", "y"):
        assert _matmul(**{k: None}) == VALUE, k
    assert _matmul(tiles=P + 8) == UNSUPPORTED
    need = S.q4_workspace_size(2048, 12288, 64)
    assert need > 0
    big = dict(rows=2048, cols=12288, ldx=12288, ldy=2048, n=64)
    assert _matmul(**big) == VALUE and b"workspace" in S.lib().spmv_last_error()
    assert _matmul(ws=P, wsb=need - 1, **big) == VALUE and _matmul(ws=P + 8, wsb=need, **big) == UNSUPPORTED
    assert _matmul(rows=0, y=None) == OK and _matmul(n=0, x=None, y=None) == OK
    assert S.lib().q4_workspace_size(4, 4, 4, None) == VALUE
    z = ctypes.c_size_t()
    for a in ((-1, 4, 4), (4, -1, 4), (4, 4, -1)):
        assert S.lib().q4_workspace_size(*a, ctypes.byref(z)) == VALUE


def test_matmul_workspace_serves_fewer_tokens():
    for rows, cols in ((64, 12288), (2048, 12288), (256, 4096), (4096, 4096), (12288, 128)):
        sizes = [S.q4_workspace_size(rows, cols, n) for n in range(0, 700)]
        assert sizes == sorted(sizes) and sizes[0] == 0


def _moe(n=4, k=2, e=8, dim=64, inter=96, group=32, zp=0, keys=P, w=None, up=P, dn=P, dt=F16, x=P, ldx=64, y=P, ydt=F16,
         ldy=64, ws=P, wsb=None):
    if wsb is None:
        z = ctypes.c_size_t()
        S.lib().moe_workspace_size(n, k, dim, inter, ctypes.byref(z))
        wsb = z.value
    return S.lib().moe_apply(n, k, e, dim, inter, group, zp, keys, w, up, dn, dt, x, ldx, y, ydt, ldy, ws, wsb, None)


def test_moe_refusals():
    assert _moe(n=-1) == VALUE and _moe(k=0) == VALUE and _moe(e=0) == VALUE
    assert _moe(dim=0) == VALUE and _moe(inter=0) == VALUE and _moe(group=20) == VALUE
    assert _moe(n=257) == UNSUPPORTED and _moe(n=256, k=17) == UNSUPPORTED and _moe(e=1025) == UNSUPPORTED
    assert _moe(dim=7, ldx=7, ldy=7) == UNSUPPORTED
    assert _moe(dt=F32) == UNSUPPORTED and _moe(dt=9) == VALUE and _moe(ydt=9) == VALUE and _moe(ydt=BF16) == UNSUPPORTED
    assert _moe(ldx=63) == VALUE and _moe(ldy=63) == VALUE
    for p in ("keys", "up", "dn", "x", "y", "ws"):
        assert _moe(**{p: None}) == VALUE, p
    assert _moe(up=P + 8) == UNSUPPORTED and _moe(dn=P + 8) == UNSUPPORTED and _moe(ws=P + 8) == UNSUPPORTED
    assert _moe(wsb=S.moe_workspace_size(4, 2, 64, 96) - 1) == VALUE
    assert b"workspace" in S.lib().spmv_last_error()
    assert _moe(dim=2 ** 24 + 1, ldx=2 ** 31, ldy=2 ** 31) == UNSUPPORTED and _moe(inter=2 ** 24 + 1) == UNSUPPORTED
    assert _moe(e=1024, n=256, k=16, inter=2 ** 24) == OVERFLOW
    assert _moe(n=0, keys=None, x=None, y=None, ws=None) == OK
    z = ctypes.c_size_t()
    L = S.lib()
    assert L.moe_workspace_size(4, 2, 64, 96, None) == VALUE and L.moe_workspace_size(-1, 2, 64, 96, ctypes.byref(z)) == VALUE
    assert L.moe_workspace_size(4, 0, 64, 96, ctypes.byref(z)) == VALUE and L.moe_workspace_size(4, 2, 64, 0, ctypes.byref(z)) == VALUE
    assert S.moe_workspace_size(0, 1, 9, 5) == 0 and L.moe_workspace_size(4, 2, 0, 8, ctypes.byref(z)) == VALUE


def _lookup(n=4, v=10, dim=8, dt=F16, ids=P, t=P, ldt=8, y=P, ydt=F16, ldy=8):
    return S.lib().embed_lookup(n, v, dim, dt, ids, t, ldt, 1.0, y, ydt, ldy, None)


def test_lookup_refusals():
    assert _lookup(n=-1) == VALUE and _lookup(v=-1) == VALUE and _lookup(dim=-1) == VALUE and _lookup(dt=3) == VALUE
    assert _lookup(ydt=3) == VALUE and _lookup(ydt=BF16) == UNSUPPORTED and _lookup(dt=F32) == UNSUPPORTED
    assert _lookup(ldt=7) == VALUE and _lookup(ldy=7) == VALUE
    assert _lookup(ids=None) == VALUE and _lookup(t=None) == VALUE and _lookup(y=None) == VALUE
    assert _lookup(n=2 ** 31 - 1, dim=2 ** 20, ldt=2 ** 20, ldy=2 ** 20) == OVERFLOW
    assert _lookup(n=0, ids=None, y=None) == OK and _lookup(dim=0, ldt=0, ldy=0, t=None) == OK


def _grad(n=40, v=10, dim=8, dt=F16, ids=P, dy=P, lddy=8, add=0, t=P, ldt=8, ws=P, wsb=None):
    if wsb is None:
        z = ctypes.c_size_t()
        S.lib().embed_grad_workspace_size(n, v, dim, ctypes.byref(z))
        wsb = z.value
    return S.lib().embed_grad(n, v, dim, dt, ids, dy, lddy, 1.0, add, t, ldt, ws, wsb, None)


def test_grad_refusals():
    assert _grad(n=-1) == VALUE and _grad(v=-1) == VALUE and _grad(dim=-1) == VALUE and _grad(dt=3) == VALUE
    assert _grad(n=2 ** 22 + 1) == UNSUPPORTED
    assert _grad(lddy=7) == VALUE and _grad(ldt=7) == VALUE
    assert _grad(ids=None) == VALUE and _grad(dy=None) == VALUE and _grad(t=None) == VALUE and _grad(ws=None) == VALUE
    assert _grad(ws=P + 8) == UNSUPPORTED
    assert _grad(wsb=S.embed_grad_workspace_size(40, 10, 8) - 1) == VALUE
    assert _grad(v=0, t=None) == OK and _grad(dim=0, lddy=0, ldt=0, dy=None) == OK
    assert _grad(n=0, add=1, ids=None, dy=None, t=None, ws=None) == OK
    assert S.lib().embed_grad_workspace_size(4, 4, 4, None) == VALUE
    assert S.embed_grad_workspace_size(0, 100, 8) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    c, s, x = torch.zeros(4, 16, dtype=torch.int32), torch.ones(4, 1).half(), torch.zeros(2, 100).half()
    with pytest.raises(TypeError):
        S.Q4Matrix(4, 100, c, s)
    with pytest.raises(ValueError):
        S.Q4Matrix(4, 100, c, s, group=100)
    with pytest.raises(TypeError):
        S.q4_matmul(4, 100, c, 1.0, x, 0.0, torch.zeros(2, 4))
    with pytest.raises(TypeError):
        S.q4_quantize(torch.zeros(4, 100), c, s)
    with pytest.raises(TypeError):
        S.embed_lookup(torch.zeros(2, dtype=torch.int32), x, x)
    with pytest.raises(TypeError):
        S.embed_grad(torch.zeros(2, dtype=torch.int32), x, torch.zeros(4, 100), None)


def test_layout_reference_round_trips():
    """The layout that the GPU tests count on, against the header's words."""
    import quant_refs as Q
    q = np.random.default_rng(0).integers(0, 16, (3, 256))
    words = Q.pack(q)
    assert np.array_equal(Q.unpack(words), q)
    w = words.numpy().view(np.uint32)
    for b, j, m, e in ((0, 0, 0, 0), (0, 3, 1, 5), (1, 2, 3, 6), (1, 1, 0, 7)):
        i = e // 2 + 4 * (e % 2)
        assert (w[1, 16 * b + 4 * j + m] >> np.uint32(4 * i)) & 15 == q[1, 128 * b + 32 * m + 8 * j + e]
