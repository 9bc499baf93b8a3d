"""Rows of a table by id and the table's gradient on the GPU against 64 bits and
against differences: repeated ids, ids outside, one id for all, sizes and types."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
import quant_refs as Q  # noqa: E402

pytestmark = pytest.mark.gpu

F = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _ids(kind, n, v, seed):
    rng = np.random.default_rng(seed)
    if kind == "mixed":
        ids = rng.integers(0, v, n)
        bad = rng.random(n) < 0.1
        ids[bad] = rng.choice([-1, v, v + 3, -2 ** 31, 2 ** 31 - 1], int(bad.sum()))
    elif kind == "one":
        ids = np.full(n, v - 1)
    elif kind == "none":
        ids = np.full(n, -1)
    elif kind == "runs":
        ids = np.repeat(rng.integers(0, v, n // 23 + 1), 23)[:n]
    else:
        ids = rng.zipf(1.4, n) % v
    return ids.astype(np.int32)


def _rows(n, width, dt, layout, gen, fill=None):
    extra, first = {"packed": (0, 0), "strided": (64, 8), "odd": (3, 1)}[layout]
    buf = torch.randn(n, width + extra, device="cuda", generator=gen)
    buf = (buf if fill is None else torch.full_like(buf, fill)).to(dt)
    return buf[:, first:first + width], buf


SHAPES = [(1, 1, 1), (1, 5, 8), (7, 3, 3), (64, 100, 64), (65, 1000, 130), (300, 50, 1111), (1000, 4097, 520),
          (33, 7, 4100)]


@pytest.mark.parametrize("dt,ydt", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("layout", ["packed", "strided", "odd"])
def test_lookup(dt, ydt, shape, layout):
    n, v, d = shape
    gen = torch.Generator(device="cuda").manual_seed(n + d)
    table, _ = _rows(v, d, F[dt], layout, gen)
    y, buf = _rows(n, d, F[ydt], layout, gen, float("nan"))
    ids = _ids("mixed", n, v, d)
    S.embed_lookup(torch.from_numpy(ids).cuda(), table, y, scale=1.7)
    ref, bound = Q.embed(ids, table, np.float32(1.7).item(), y.dtype)
    R.check(y, ref, bound)
    assert int(torch.isnan(buf).sum()) == buf.numel() - n * d          # nothing beside the rows


def test_lookup_of_nothing():
    y = torch.full((4, 8), 5.0, device="cuda")
    S.embed_lookup(torch.zeros(4, dtype=torch.int32, device="cuda"), torch.empty(0, 8, device="cuda"), y)
    assert (y == 0).all()
    S.embed_lookup(torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(3, 8, device="cuda"), y[:0])


def test_lookup_keeps_infinities():
    t = torch.tensor([[1.0, float("inf"), float("nan"), -0.0] * 4], device="cuda").half()
    y = S.embed_lookup(torch.zeros(2, dtype=torch.int32, device="cuda"), t, torch.empty(2, 16, device="cuda").half(), 2.0)
    assert torch.equal(torch.isnan(y), torch.isnan(t).expand(2, -1)) and (y[:, 1] == float("inf")).all() and (y[:, 0] == 2).all()


def _grad(ids, dy, v, scale, first, layout="packed", gen=None):
    n, d = dy.shape
    out, buf = _rows(v, d, torch.float32, layout, gen or torch.Generator(device="cuda"), float("nan"))
    if first is not None:
        out.copy_(first)
    ws = torch.empty(S.embed_grad_workspace_size(n, v, d), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    S.embed_grad(torch.from_numpy(ids).cuda(), dy, out, ws, scale=scale, accumulate=first is not None)
    assert int(torch.isnan(buf).sum()) == buf.numel() - v * d
    return out


@pytest.mark.parametrize("kind", ["mixed", "one", "none", "runs", "skewed"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (15, 4, 8), (16, 3, 3), (17, 3, 12), (64, 1, 64), (100, 5000, 130), (700, 50, 1111),
                                   (3000, 4097, 72), (20000, 300, 24), (70000, 70000, 8)])
@pytest.mark.parametrize("add", [False, True])
def test_grad(kind, shape, add):
    n, v, d = shape
    gen = torch.Generator(device="cuda").manual_seed(n + v)
    dt = ["f16", "bf16", "f32"][(n + d) % 3]
    dy = torch.randn(n, d, device="cuda", generator=gen).to(F[dt])
    first = torch.randn(v, d, device="cuda", generator=gen) if add else None
    ids = _ids(kind, n, v, seed=n)
    out = _grad(ids, dy, v, 1.7, first)
    ref, bound = Q.embed_grad(ids, dy, v, np.float32(1.7).item(), first)
    R.check(out, ref, bound, f"{kind} {shape} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["strided", "odd"])
@pytest.mark.parametrize("d", [1, 3, 4, 7, 8, 9, 257, 1000])
@pytest.mark.parametrize("add", [False, True])
def test_grad_strides_and_widths(dt, layout, d, add):
    n, v = 130, 37
    gen = torch.Generator(device="cuda").manual_seed(d)
    dy, _ = _rows(n, d, F[dt], layout, gen)
    first = torch.randn(v, d, device="cuda", generator=gen) if add else None
    ids = _ids("skewed", n, v, seed=d)
    ids[5] = -1
    dy[5] = float("nan")                                     # a row that is not read
    out = _grad(ids, dy, v, -0.5, first, layout, gen)
    dy[5] = 0.0
    ref, bound = Q.embed_grad(ids, dy, v, -0.5, first)
    R.check(out, ref, bound)


@pytest.mark.parametrize("n", [50, 16384, 16385, 33000])
def test_grad_bits_repeat_and_the_sort_is_stable(n):
    """Every row is the sum in the tokens' order: a table of one column shows it."""
    ids = _ids("skewed", n, 900, seed=n)
    dy = torch.randn(n, 16, device="cuda")
    a = _grad(ids, dy, 900, 1.0, None)
    assert torch.equal(a, _grad(ids, dy, 900, 1.0, None))
    # positions within a row's own run decide: with tokens of other rows moved around it stays the same
    counts = np.bincount(ids, minlength=900)
    few = np.flatnonzero((counts > 0) & (counts <= 2))
    d64 = R.f64(dy)
    for v in few[:50]:
        at = np.flatnonzero(ids == v)
        s = dy[at[0]].clone()
        if len(at) == 2:
            s = s + dy[at[1]]
        assert torch.equal(a[v], s), v
    assert d64.shape[0] == n


def test_grad_of_nothing():
    out = torch.full((5, 6), 3.0, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    dy = torch.empty(0, 6, device="cuda")
    S.embed_grad(e, dy, out, None, accumulate=True)
    assert (out == 3.0).all()
    S.embed_grad(e, dy, out, None)
    assert (out == 0.0).all()
    S.embed_grad(torch.zeros(3, dtype=torch.int32, device="cuda"), torch.empty(3, 6, device="cuda"), out[:0],
                 torch.empty(S.embed_grad_workspace_size(3, 0, 6), dtype=torch.uint8, device="cuda"))


def test_grad_against_differences():
    """d/dE of sum(lookup(E) * g), by differences of the lookup in fp32 with exact steps."""
    ids = np.array([2, 0, 2, -1, 4, 2], np.int32)
    t, di = torch.from_numpy(ids).cuda(), 6
    table = torch.randint(-8, 9, (5, di), device="cuda").float() / 8
    g = torch.randint(-8, 9, (6, di), device="cuda").float() / 8
    grad = _grad(ids, g, 5, 0.5, None)
    look = lambda e: (S.embed_lookup(t, e, torch.empty(6, di, device="cuda"), 0.5) * g).sum().item()  # noqa: E731
    for v in range(5):
        for j in range(di):
            a, b = table.clone(), table.clone()
            a[v, j] += 0.25
            b[v, j] -= 0.25
            assert (look(a) - look(b)) / 0.5 == grad[v, j].item()


def test_refusals():
    ids, table, y = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(9, 16, device="cuda").half(), torch.zeros(4, 16, device="cuda")
    for i, t, o in ((ids, table, y[:3]), (ids, table, y[:, :15]), (ids[::2], table, y[:2]), (ids, table[0], y), (ids, table.t(), y)):
        with pytest.raises(ValueError):
            S.embed_lookup(i, t, o)
    for i, t, o in ((ids.long(), table, y), (ids, table.double(), y), (ids, table, y.bfloat16()), (ids, table.cpu(), y)):
        with pytest.raises(TypeError):
            S.embed_lookup(i, t, o)
    dy, ws = torch.zeros(4, 16, device="cuda"), torch.empty(S.embed_grad_workspace_size(4, 9, 16), dtype=torch.uint8, device="cuda")
    dt = torch.zeros(9, 16, device="cuda")
    for i, d, o in ((ids[:3], dy, dt), (ids, dy, dt[:, :15]), (ids, dy, dt[0]), (ids, dy.t(), dt)):
        with pytest.raises(ValueError):
            S.embed_grad(i, d, o, ws)
    for i, d, o in ((ids.long(), dy, dt), (ids, dy, dt.half()), (ids, dy.double(), dt)):
        with pytest.raises(TypeError):
            S.embed_grad(i, d, o, ws)
    for bad in (None, ws[:-16]):
        with pytest.raises(S.SpmvError):
            S.embed_grad(ids, dy, dt, bad)


def test_captured_and_replayed():
    n, v, d = 500, 90, 128
    ids, dy = torch.from_numpy(_ids("skewed", n, v, 1)).cuda(), torch.randn(n, d, device="cuda").bfloat16()
    out = torch.empty(v, d, device="cuda")
    ws = torch.empty(S.embed_grad_workspace_size(n, v, d), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S.embed_grad(ids, dy, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.embed_grad(ids, dy, out, ws)
    for i in range(3):
        new = _ids(["mixed", "one", "runs"][i], n, v, 40 + i)
        ids.copy_(torch.from_numpy(new))
        dy.copy_(torch.randn(n, d, device="cuda"))
        out.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        _grad(_ids("mixed", 77, v, i), dy[:77], v, 1.0, None)
        torch.cuda.synchronize()
        assert torch.equal(out, _grad(new, dy, v, 1.0, None)), i
