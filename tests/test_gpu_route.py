"""Tokens sorted by group and back on the GPU: the plan against a stable NumPy
sort (exactly), the row movements and their gradients against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402

pytestmark = pytest.mark.gpu

F = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _keys(kind, n, k, e, seed):
    rng = np.random.default_rng(seed)
    if kind == "mixed":
        keys = rng.integers(0, e, (n, k))
        keys[rng.random((n, k)) < 0.1] = rng.choice([-1, e, e + 5, -2 ** 31, 2 ** 31 - 1])
    elif kind == "uniform":
        keys = rng.integers(0, e, (n, k))
    elif kind == "one":
        keys = np.full((n, k), e - 1)            # every slot, twice and more per token, in one group
    elif kind == "none":
        keys = np.full((n, k), -1)
    else:
        keys = np.sort(rng.zipf(1.3, (n, k)) % e, axis=1)
    return keys.astype(np.int32)


def _plan(keys, e):
    n, k = keys.shape
    p = S.RoutePlan(n, k, e)
    for t in (p.offsets, p.order, p.pos, p.tiles):
        t.fill_(-77)
    p.workspace.fill_(255)
    return p.build(torch.from_numpy(keys).cuda())


PLANS = [(0, 1, 3), (1, 1, 1), (1, 4, 2), (5, 2, 8), (64, 2, 8), (65, 3, 200), (4096, 2, 16), (2731, 3, 64),
         (8193, 1, 7), (5000, 8, 64), (3000, 4, 1500), (2500, 1, 2048), (300, 2, 895), (300, 2, 896), (20000, 1, 895)]


@pytest.mark.parametrize("shape", PLANS)
@pytest.mark.parametrize("kind", ["mixed", "one", "none", "skewed"])
def test_plan(shape, kind):
    n, k, e = shape
    keys = _keys(kind, n, k, e, seed=n + k)
    p = _plan(keys, e)
    offsets, order, pos, tiles = R.route_plan(keys, e)
    assert p.offsets.cpu().tolist() == offsets.tolist()
    assert np.array_equal(p.order.cpu().numpy(), order)
    assert np.array_equal(p.pos.cpu().numpy().reshape(-1), pos)
    got = p.tiles.cpu().numpy()
    assert [tuple(t) for t in got[:len(tiles)].tolist()] == [tuple(int(v) for v in t) for t in tiles]
    assert (got[len(tiles):] == [-1, 0, 0, 0]).all()


DATA = [(1, 1, 1, 8), (7, 2, 3, 1), (64, 2, 8, 4096), (333, 3, 13, 1111), (100, 9, 20, 520), (50, 17, 4, 2056),
        (2000, 8, 32, 72)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", DATA)
@pytest.mark.parametrize("layout", ["packed", "strided", "odd"])
def test_rows_there_and_back(shape, dt, layout):
    n, k, e, d = shape
    t = F[dt]
    keys = _keys("mixed", n, k, e, seed=d)
    p = _plan(keys, e)
    offsets, order, pos, _ = R.route_plan(keys, e)
    m = int(offsets[-1])
    gen = torch.Generator(device="cuda").manual_seed(n * d)

    def rows(r, fill=None):
        """[r, d] in a wider buffer: rows of their own, 64 elements apart, or an odd stride and offset."""
        extra, first = {"packed": (0, 0), "strided": (64, 8), "odd": (3, 1)}[layout]
        buf = torch.randn(r, d + extra, device="cuda", generator=gen)
        buf = (buf if fill is None else torch.full_like(buf, fill)).to(t)
        if layout == "strided":
            first = 0
        return buf[:, first:first + d]

    w = torch.rand(n, k, device="cuda", generator=gen) * 2 - 0.5
    x, ys, dy = rows(n), rows(n * k), rows(n)
    order_t = torch.from_numpy(order)
    tok = order_t[:m] // k
    x64, ys64, dy64, w64 = R.f64(x), R.f64(ys), R.f64(dy), R.f64(w).reshape(-1)

    xs = rows(n * k, -3.0)
    assert p.gather(x, xs) is xs
    assert torch.equal(R.f64(xs)[:m], x64[tok]) and (R.f64(xs)[m:] == -3.0).all()
    p.gather(x, xs, w)
    ref = x64[tok] * w64[order_t[:m], None]
    R.check(xs[:m], ref, ref.abs() * 2.0 ** -24 + R.rounded(ref, t), "weighted gather")
    assert (R.f64(xs)[m:] == -3.0).all()

    for weights in (w, None):
        ref = torch.zeros(n, d, dtype=torch.float64)
        mag = torch.zeros(n, d, dtype=torch.float64)
        f = w64 if weights is not None else torch.ones(n * k, dtype=torch.float64)
        ref.index_add_(0, tok, ys64[:m] * f[order_t[:m], None])
        mag.index_add_(0, tok, (ys64[:m] * f[order_t[:m], None]).abs())
        y = rows(n, float("nan"))
        p.combine(ys, y, weights)
        R.check(y, ref, mag * (k * 2.0 ** -24) + R.rounded(ref.abs() + mag * (k * 2.0 ** -24), t), "combine")

        dys, dw = rows(n * k, -3.0), torch.full((n, k), float("nan"), device="cuda")
        p.combine_grad(dy, ys, weights, dys, dw)
        gref = dy64[tok] * f[order_t[:m], None]
        R.check(dys[:m], gref, gref.abs() * 2.0 ** -24 + R.rounded(gref, t), "dys")
        assert (R.f64(dys)[m:] == -3.0).all()
        dref, dmag = torch.zeros(n * k, dtype=torch.float64), torch.zeros(n * k, dtype=torch.float64)
        dref[order_t[:m]] = (ys64[:m] * dy64[tok]).sum(1)
        dmag[order_t[:m]] = (ys64[:m] * dy64[tok]).abs().sum(1)
        R.check(dw.reshape(-1), dref, dmag * ((d + 2) * 2.0 ** -24), "dw")


def test_combine_gradient_is_the_difference_quotient():
    """<dy, y> is linear in w and in ys: steps of a power of two give its
    derivatives up to the rounding of y."""
    n, k, e, d = 40, 3, 5, 96
    keys = _keys("mixed", n, k, e, 3)
    p = _plan(keys, e)
    g = torch.Generator(device="cuda").manual_seed(5)
    ys, dy = (torch.randn(r, d, device="cuda", generator=g) for r in (n * k, n))
    w = torch.rand(n, k, device="cuda", generator=g)
    dys, dw = torch.zeros_like(ys), torch.zeros_like(w)
    p.combine_grad(dy, ys, w, dys, dw)
    vw = torch.randint(-4, 5, w.shape, device="cuda", generator=g).float()
    vy = torch.randint(-4, 5, ys.shape, device="cuda", generator=g).float()
    run = lambda a, b: R.f64(p.combine(a, torch.empty_like(dy), b))  # noqa: E731
    dy64 = R.f64(dy)
    for up, down, want in ((run(ys, w + vw), run(ys, w - vw), (R.f64(dw) * R.f64(vw)).sum()),
                           (run(ys + vy, w), run(ys - vy, w), (R.f64(dys) * R.f64(vy)).sum())):
        got = ((up - down) / 2 * dy64).sum()
        # each y, and w +- v or ys +- v, is rounded in fp32: values up to 4 + 5, k of them
        tol = (dy64.abs().sum() * 9 * 9 * k * (k + 3) * 2.0 ** -24)
        assert abs(got - want) <= tol


def test_graph_replays_and_second_stream():
    n, k, e, d = 700, 2, 12, 264
    keys = torch.from_numpy(_keys("mixed", n, k, e, 1)).cuda()
    p, q = S.RoutePlan(n, k, e), S.RoutePlan(n, k, e)
    x = torch.randn(n, d, device="cuda").bfloat16()
    w = torch.rand(n, k, device="cuda")
    xs, y = torch.zeros(n * k, d, device="cuda", dtype=x.dtype), torch.zeros_like(x)
    dys, dw = torch.zeros_like(xs), torch.zeros_like(w)

    def step(p):
        p.build(keys)
        p.gather(x, xs)
        p.combine(xs, y, w)
        p.combine_grad(x, xs, w, dys, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(p)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(p)
    for i in range(4):
        keys.copy_(torch.from_numpy(_keys("mixed" if i != 2 else "none", n, k, e, 10 + i)))
        x.copy_(torch.randn(n, d, device="cuda"))
        torch.cuda.synchronize()
        for t in (xs, y, dys, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (p.offsets, p.order, p.pos, p.tiles, xs, y, dys, dw)]
        for t in (xs, y, dys, dw):
            t.zero_()
        step(q)
        torch.cuda.synchronize()
        want = [q.offsets, q.order, q.pos, q.tiles, xs, y, dys, dw]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_refusals_of_shapes():
    p = S.RoutePlan(4, 2, 3)
    x = torch.zeros(4, 8, device="cuda")
    xs = torch.zeros(8, 8, device="cuda")
    with pytest.raises(ValueError):
        p.gather(x, xs[:7])
    with pytest.raises(TypeError):
        p.gather(x, xs.half())
    with pytest.raises(ValueError):
        p.gather(x.t().contiguous().t(), xs)
    with pytest.raises(ValueError):
        p.gather(x[:1].expand(4, 8), xs)
    with pytest.raises(TypeError):
        p.gather(x.int(), xs.int())
    with pytest.raises(ValueError):
        p.combine(xs, x, torch.ones(4, 1, device="cuda"))
    with pytest.raises(TypeError):
        p.build(torch.zeros(8, dtype=torch.int64, device="cuda"))
    with pytest.raises(S.SpmvError):
        S.route_plan(3, torch.zeros(1 << 16, dtype=torch.int32, device="cuda"),
                     *(torch.zeros(1 << 18, dtype=torch.int32, device="cuda") for _ in range(4)))
