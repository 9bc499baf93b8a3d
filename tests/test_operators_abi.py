"""CPU-side checks of the many-token operators' C entry points (no kernel is
launched): sizes, refusals with their statuses, and the calls that have
nothing to do."""
import ctypes

import numpy as np
import pytest

import sparse_matrix_vector_amd as S

OK, VALUE, OVERFLOW, UNSUPPORTED = 0, 1, 4, 5
P = 4096                                     # a pointer that is aligned and never followed


def test_tile_count_bounds_every_plan():
    rng = np.random.default_rng(0)
    for _ in range(400):
        n, g = int(rng.integers(0, 300)), int(rng.integers(1, 40))
        keys = rng.integers(0, g + 1, n) if rng.random() < 0.7 else np.full(n, rng.integers(0, g + 1))
        used = sum(-(-int(c) // 16) for c in np.bincount(keys, minlength=g + 1))
        assert used <= S.route_tile_count(n, g)
    # every bin one row past a tile
    for g in (1, 7, 100):
        n = (g + 1) * 17
        assert 2 * (g + 1) <= S.route_tile_count(n, g)
    assert S.route_tile_count(0, 5) == 0 and S.route_tile_count(1, 5) == 1


def test_route_sizes_and_refusals():
    L = S.lib()
    n, z = ctypes.c_int32(), ctypes.c_size_t()
    assert L.route_tile_count(-1, 4, ctypes.byref(n)) == VALUE
    assert L.route_tile_count(4, 0, ctypes.byref(n)) == VALUE
    assert L.route_tile_count(4, 4, None) == VALUE
    assert L.route_tile_count(4, 2049, ctypes.byref(n)) == UNSUPPORTED
    assert L.route_tile_count((1 << 22) + 1, 4, ctypes.byref(n)) == UNSUPPORTED
    assert L.route_workspace_size(4, 4, None) == VALUE
    assert L.route_workspace_size(-1, 4, ctypes.byref(z)) == VALUE
    assert S.route_workspace_size(100, 8) == 0
    big = S.route_workspace_size(1 << 20, 8)
    assert big > 0
    assert L.route_plan(1 << 20, 8, P, P, P, P, P, None, 0, None) == VALUE          # no workspace
    assert L.route_plan(1 << 20, 8, P, P, P, P, P, P, big - 1, None) == VALUE       # too small
    assert L.route_plan(1 << 20, 8, P, P, P, P, P, P + 2, big, None) == UNSUPPORTED
    assert L.route_plan(8, 8, P, P, P, P, P + 4, None, 0, None) == UNSUPPORTED      # tiles not 16-byte aligned
    for k in range(5):                                                              # each NULL in turn
        a = [P] * 5
        a[k] = None
        assert L.route_plan(8, 8, *a, None, 0, None) == VALUE, k
    assert L.route_plan(8, 0, P, P, P, P, P, None, 0, None) == VALUE


def test_route_data_refusals():
    L = S.lib()
    def gather(n=4, k=2, dim=8, dt=0, pos=P, w=None, x=P, ldx=8, xs=P, ldxs=8):
        return L.route_gather(n, k, dim, dt, pos, w, x, ldx, xs, ldxs, None)
    assert gather(n=-1) == VALUE and gather(k=0) == VALUE and gather(dim=-1) == VALUE and gather(dt=3) == VALUE
    assert gather(ldx=7) == VALUE and gather(ldxs=7) == VALUE
    assert gather(pos=None) == VALUE and gather(xs=None) == VALUE and gather(x=None) == VALUE
    assert gather(n=1 << 30, k=4) == OVERFLOW
    assert gather(n=0, x=None, xs=None, pos=None) == OK
    assert gather(dim=0, ldx=0, ldxs=0, x=None, xs=None) == OK

    def combine(n=4, k=2, dim=8, dt=0, pos=P, w=None, ys=P, ldys=8, y=P, ldy=8):
        return L.route_combine(n, k, dim, dt, pos, w, ys, ldys, y, ldy, None)
    assert combine(n=-1) == VALUE and combine(dt=-1) == VALUE and combine(ldy=7) == VALUE and combine(ldys=7) == VALUE
    assert combine(pos=None) == VALUE and combine(ys=None) == VALUE and combine(y=None) == VALUE
    assert combine(n=0, pos=None) == OK

    def grad(n=4, k=2, dim=8, dt=0, dy=P, lddy=8, ys=P, ldys=8, pos=P, w=P, dys=P, lddys=8, dw=P):
        return L.route_combine_grad(n, k, dim, dt, dy, lddy, ys, ldys, pos, w, dys, lddys, dw, None)
    assert grad(k=0) == VALUE and grad(lddy=7) == VALUE and grad(ldys=7) == VALUE and grad(lddys=7) == VALUE
    assert grad(dw=None) == VALUE and grad(dy=None) == VALUE and grad(pos=None) == VALUE
    assert grad(n=0, pos=None, dw=None) == OK


def _lora(fn="lora_apply", **kw):
    a = dict(n=20, n_in=64, n_out=32, ad=3, r=8, ranks=None, scale=None, A=P, B=P, dt=0, order=P, off=P, tiles=P,
             nt=None, x=P, ldx=64, yin=P, ldyin=32, y=2 * P, ydt=2, ldy=32, ws=P, wsb=None)
    a.update(kw)
    if a["nt"] is None:
        a["nt"] = S.route_tile_count(a["n"], a["ad"]) if 0 <= a["n"] and 1 <= a["ad"] <= 2048 else 0
    if a["wsb"] is None:
        a["wsb"] = S.lora_workspace_size(a["n"], a["r"]) if a["n"] >= 0 and 1 <= a["r"] <= 128 else 0
    head = [a[k] for k in ("n", "n_in", "n_out", "ad", "r", "ranks", "scale", "A", "B", "dt", "order", "off", "tiles",
                           "nt", "x", "ldx")]
    if fn == "lora_apply":
        tail = [a[k] for k in ("yin", "ldyin", "y", "ydt", "ldy", "ws", "wsb")]
    else:
        tail = [a["yin"], a["ldyin"], a.get("dA", P), a.get("dB", P), a["ws"], a["wsb"]]
    return getattr(S.lib(), fn)(*head, *tail, None)


@pytest.mark.parametrize("fn", ["lora_apply", "lora_grad"])
def test_lora_refusals(fn):
    call = lambda **kw: _lora(fn, **kw)  # noqa: E731
    assert call(n=-1) == VALUE and call(n_in=0) == VALUE and call(n_out=0) == VALUE and call(ad=0) == VALUE
    assert call(r=0) == VALUE and call(r=129) == UNSUPPORTED and call(ad=2049) == UNSUPPORTED
    assert call(dt=2) == UNSUPPORTED and call(dt=7) == VALUE
    assert call(nt=1) == VALUE                                  # tiles of another plan
    assert b"tiles" in S.lib().spmv_last_error()
    assert call(A=None) == VALUE and call(B=None) == VALUE and call(order=None) == VALUE
    assert call(off=None) == VALUE and call(tiles=None) == VALUE and call(x=None) == VALUE
    assert call(tiles=P + 8) == UNSUPPORTED
    assert call(ws=None) == VALUE and call(wsb=16) == VALUE and call(ws=P + 8) == UNSUPPORTED
    assert call(ldx=63) == VALUE and call(ldyin=31) == VALUE


def test_lora_apply_refusals_of_y():
    assert _lora(ydt=1) == UNSUPPORTED and _lora(ydt=9) == VALUE and _lora(dt=1, ydt=0) == UNSUPPORTED
    assert _lora(ldy=31) == VALUE and _lora(y=None) == VALUE
    assert _lora(yin=2 * P, ldyin=40) == VALUE                  # in place with another stride
    assert _lora(n=0, x=None, y=None, yin=None, order=None, tiles=None, ws=None) == OK
    assert _lora("lora_grad", dA=None) == VALUE and _lora("lora_grad", dB=None) == VALUE
    assert S.lib().lora_workspace_size(4, 8, None) == VALUE
    z = ctypes.c_size_t()
    assert S.lib().lora_workspace_size(-1, 8, ctypes.byref(z)) == VALUE
    assert S.lib().lora_workspace_size(4, 0, ctypes.byref(z)) == VALUE
    assert S.lib().lora_workspace_size(4, 129, ctypes.byref(z)) == UNSUPPORTED


def _spmm(i8=False, **kw):
    a = dict(g=1, rows=32, cols=64, b=4, mrp=P, codes=P, vals=P, scale=P, plan=P, off=None, n=4, x=P, ldx=64, y=P,
             ydt=2, ldy=32, ws=None, wsb=0)
    a.update(kw)
    head = [a[k] for k in ("g", "rows", "cols", "b", "mrp", "codes", "vals")] + ([a["scale"]] if i8 else [])
    return getattr(S.lib(), "macko_spmm_i8" if i8 else "macko_spmm")(
        *head, a["plan"], a["off"], a["n"], 1.0, a["x"], a["ldx"], 0.0, a["y"], a["ydt"], a["ldy"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("i8", [False, True])
def test_spmm_refusals(i8):
    call = lambda **kw: _spmm(i8, **kw)  # noqa: E731
    assert call(g=0) == VALUE and call(n=-1) == VALUE and call(rows=-1) == VALUE and call(cols=-1) == VALUE
    assert call(b=3) == VALUE and call(ydt=1) == UNSUPPORTED and call(ydt=5) == VALUE
    assert call(cols=(1 << 20) + 1, ldx=1 << 21) == UNSUPPORTED
    assert call(rows=16 * 65535 + 1, ldy=1 << 21) == UNSUPPORTED and call(g=4096, off=P) == UNSUPPORTED
    assert call(g=4095, rows=600000, ldy=600000, off=P) == OVERFLOW
    assert call(ldx=63) == VALUE and call(ldy=31) == VALUE
    assert call(g=2) == VALUE                                   # several groups without offsets
    for k in ("mrp", "codes", "vals", "plan", "x", "y"):
        assert call(**{k: None}) == VALUE, k
    assert call(cols=0, ldx=0) == VALUE
    assert call(vals=P + 4) == UNSUPPORTED and call(codes=P + 2) == UNSUPPORTED and call(b=8, codes=P + 4) == UNSUPPORTED
    # x that needs packing: no workspace, too small, misaligned
    need = S.macko_spmm_workspace_size(1, 32, 64, 4)
    assert need == 4 * 64 * 2 and S.macko_spmm_workspace_size(1, 32, 9, 3) == 3 * 16 * 2
    for kw in (dict(x=P + 2), dict(ldx=65), dict(cols=63, ldx=64)):
        assert call(**kw) == VALUE
        assert b"workspace" in S.lib().spmv_last_error()
        assert call(ws=P, wsb=need - 1, **kw) == VALUE and call(ws=P + 8, wsb=need, **kw) == VALUE
    if i8:
        assert call(scale=None) == VALUE
    assert call(rows=0, ldy=0, mrp=None) == OK and call(n=0, x=None, y=None) == OK


def test_spmm_plan_sizes_and_refusals():
    L = S.lib()
    z = ctypes.c_size_t()
    assert S.macko_spmm_plan_size(10, 256) == 10 * 2 * 4 and S.macko_spmm_plan_size(10, 257) == 10 * 3 * 4
    assert S.macko_spmm_plan_size(0, 100) == 0
    assert L.macko_spmm_plan_size(-1, 4, ctypes.byref(z)) == VALUE and L.macko_spmm_plan_size(4, 4, None) == VALUE
    assert L.macko_spmm_plan_size(4, (1 << 20) + 1, ctypes.byref(z)) == UNSUPPORTED
    assert L.macko_spmm_workspace_size(1, 4, 4, -1, ctypes.byref(z)) == VALUE
    assert L.macko_spmm_workspace_size(0, 4, 4, 1, ctypes.byref(z)) == VALUE
    assert L.macko_spmm_workspace_size(1, 4, 4, 1, None) == VALUE
    assert L.macko_spmm_plan(8, 64, 5, P, P, P, 1 << 20, None) == VALUE
    assert L.macko_spmm_plan(8, 64, 4, P, P, P, 8, None) == VALUE
    assert L.macko_spmm_plan(8, 64, 4, None, P, P, 1 << 20, None) == VALUE
    assert L.macko_spmm_plan(8, 0, 4, P, P, P, 1 << 20, None) == VALUE
    assert L.macko_spmm_plan(8, 64, 8, P, P + 4, P, 1 << 20, None) == UNSUPPORTED
    assert L.macko_spmm_plan(8, 64, 4, P, P, P + 2, 1 << 20, None) == UNSUPPORTED
    assert L.macko_spmm_plan(0, 64, 4, None, None, None, 0, None) == OK


def test_binding_refuses_cpu_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        S.route_combine(x, torch.zeros(4, 2, dtype=torch.int32), x)
    with pytest.raises(ValueError):
        S.route_combine(x, torch.zeros(8, dtype=torch.int32), x)
    with pytest.raises(TypeError):
        S.lora_apply(None, None, x, x, x, x, x, x, None, x, None)
    with pytest.raises(ValueError):
        S.RoutePlan(4, 2, 3, device="cpu").build(torch.zeros(7, dtype=torch.int32))
