"""The MACKO product of many tokens on the GPU against the dense product in 64
bits: code widths, int8 values, odd sizes and strides, empty and full rows,
groups of tokens, and the plan against the decoded columns."""
import numpy as np
import pytest

import gen
import oracle
from helpers import dev, host

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _weight(rows, cols, kind, b, seed, i8=False):
    """(mrow_ptr, codes, values, scales, dense float64), by the library's encoder."""
    rng = np.random.default_rng(seed)
    if kind == "ragged":                       # from empty to full rows
        lens = rng.integers(0, cols + 1, rows)
        lens[::5] = 0
        lens[1::7] = cols
    elif kind == "sparse":
        lens = np.minimum(rng.integers(0, 4, rows), cols)
    else:
        lens = np.full(rows, max(1, int(cols * (1 - float(kind)))))
    ci = np.concatenate([np.sort(rng.permutation(cols)[:n]) for n in lens]).astype(np.int32)
    rp = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    v = rng.uniform(-1, 1, len(ci)).astype(np.float16)
    v[v == 0] = np.float16(0.5)
    mrp, codes, mv = S.macko_encode(rows, cols, rp, ci, v.view(np.uint16), bdelta=b)
    q, sc = S.macko_quantize_i8(rows, mrp, mv) if i8 else (None, None)
    columns = oracle.macko_decode(mrp, codes, b)
    dense = np.zeros((rows, cols + 1))
    row = np.repeat(np.arange(rows), np.diff(mrp))
    vals = mv.view(np.float16).astype(np.float64) if not i8 else q.astype(np.float64) * sc.astype(np.float64)[row]
    np.add.at(dense, (row, np.minimum(columns, cols)), vals)
    return mrp, codes, (q if i8 else mv.view(np.float16)), sc, torch.from_numpy(dense[:, :cols])


def _matrix(w, rows, cols, b, groups=1):
    mrp, codes, vals, sc, _ = w
    one = lambda a, d: dev(a) if len(a) else torch.zeros(16, dtype=d, device="cuda")  # noqa: E731
    return S.MackoMatrix(rows, cols, dev(mrp), one(codes.view(np.int32), torch.int32),
                         one(vals, torch.int8 if sc is not None else torch.float16), None if sc is None else dev(sc),
                         n_groups=groups, bdelta=b)


def _x(T, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, cols, device="cuda", generator=g).half()


SHAPES = [(1, 1, 1), (16, 256, 16), (37, 1000, 5), (5, 17, 3), (130, 2049, 33), (64, 4096, 64), (33, 264, 100),
          (48, 255, 2), (100, 513, 129), (17, 2056, 1)]


@pytest.mark.parametrize("b", [1, 2, 4, 8])
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_product(shape, b, i8):
    rows, cols, T = shape
    for kind in ("ragged", "0.5", "0.95"):
        w = _weight(rows, cols, kind, b, rows + cols, i8)
        m = _matrix(w, rows, cols, b)
        x = _x(T, cols, 3)
        ws = m.workspace(T)
        for ydt, alpha, beta in ((torch.float32, 1.0, 0.0), (torch.float16, -0.75, 0.5)):
            y0 = torch.randn(T, rows, device="cuda").to(ydt)
            y = y0.clone() if beta else torch.full_like(y0, NAN)
            m.apply(x, y, alpha, beta, workspace=ws)
            ref, bound = R.spmm(w[4], x, alpha, beta, y0, ydt)
            R.check(y, ref, bound, f"{shape} b={b} i8={i8} {kind}")


@pytest.mark.parametrize("b", [1, 2, 4, 8])
@pytest.mark.parametrize("kind", ["ragged", "sparse", "0.5", "0.98"])
def test_plan_words(b, kind):
    """Every word names the unit that holds the first entry at or past the
    slab's start, and the column before that unit."""
    rows, cols = 61, 3001
    w = _weight(rows, cols, kind, b, 5)
    m = _matrix(w, rows, cols, b)
    mrp, codes = w[0], w[1]
    columns = oracle.macko_decode(mrp, codes, b)
    slabs = -(-cols // 256)
    plan = host(m.plan).view(np.uint32).reshape(rows, slabs + 1)
    for r in range(rows):
        c = columns[mrp[r]:mrp[r + 1]]
        for k in range(slabs + 1):
            first = int(np.searchsorted(c, 256 * k))
            unit = first // 8
            if first == len(c):
                assert plan[r, k] == len(c) // 8
            else:
                before = c[8 * unit - 1] if unit else -1
                assert plan[r, k] & 0x3FFFF == unit and plan[r, k] >> 18 == 256 * k - 1 - before, (r, k)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200, 513])
def test_token_counts(T):
    rows, cols = 160, 1536
    w = _weight(rows, cols, "0.7", 4, 8)
    m = _matrix(w, rows, cols, 4)
    x = _x(T, cols, T)
    for ydt in (torch.float32, torch.float16):
        yb = torch.full((T + 2, rows), -7.0, device="cuda", dtype=ydt)
        m.apply(x, yb[1:T + 1])
        ref, bound = R.spmm(w[4], x, 1.0, 0.0, None, ydt)
        R.check(yb[1:T + 1], ref, bound, f"T={T}")
        assert (yb[0] == -7).all() and (yb[T + 1] == -7).all()


@pytest.mark.parametrize("shape", [(64, 2304, 20), (200, 5000, 40), (1000, 2560, 300), (70, 12288, 65), (33, 8000, 24)])
@pytest.mark.parametrize("i8", [False, True])
def test_columns_split_over_workgroups(shape, i8):
    """Few rows and many columns: partial sums in the workspace (but for the
    first shape), joined in order (same bits on every call)."""
    rows, cols, T = shape
    w = _weight(rows, cols, "0.8", 4, 8, i8)
    m = _matrix(w, rows, cols, 4)
    assert (S.macko_spmm_workspace_size(1, rows, cols, T) > S.macko_spmm_workspace_size(1, rows, cols, 1) * T) == (T != 20)
    x = _x(T, cols, T)
    y0 = torch.randn(T, rows, device="cuda").half()
    ys = []
    for fill in (255, 0):
        ws = m.workspace(T).fill_(fill)
        y = y0.clone()
        m.apply(x, y, 0.5, -2.0, workspace=ws)
        ys.append(y)
    ref, bound = R.spmm(w[4], x, 0.5, -2.0, y0, torch.float16)
    R.check(ys[0], ref, bound, "split")
    assert torch.equal(*ys)


def test_split_groups_and_streams():
    """Two groups, columns split, on a stream of its own with a workspace of its own."""
    groups, rows, cols, T = 2, 96, 4096, 50
    w = _weight(groups * rows, cols, "0.8", 4, 9, True)
    m = _matrix(w, rows, cols, 4, groups)
    x = _x(T, cols, 2)
    off = torch.tensor([0, 19, 50], dtype=torch.int32, device="cuda")
    y = torch.zeros(T, rows, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    m.apply(x, y, tok_offsets=off, stream=side)
    side.synchronize()
    for g, a, b in ((0, 0, 19), (1, 19, 50)):
        ref, bound = R.spmm(w[4][g * rows:(g + 1) * rows], x[a:b], 1.0, 0.0, None, torch.float32)
        R.check(y[a:b], ref, bound, f"group {g}")


def test_full_size_against_the_vector_product():
    """12288 x 12288 at 50 %: each token against macko_spmv, same bound for both."""
    W = gen.pruned_weight(0.5, seed=3)
    enc = S.macko_encode(W.n_rows, W.n_cols, W.row_ptr, W.col_idx, W.vals_f16)
    d = [dev(enc[0]), dev(enc[1].view(np.int32)), dev(enc[2].view(np.float16))]
    m = S.MackoMatrix(W.n_rows, W.n_cols, *d)
    x = _x(20, W.n_cols, 1)
    y = torch.empty(20, W.n_rows, device="cuda")
    m.apply(x, y)
    for t in (0, 7, 15, 16, 19):
        one = torch.empty(W.n_rows, device="cuda")
        S.macko_spmv(W.n_rows, W.n_cols, *d, 1.0, x[t].contiguous(), 0.0, one)
        yr, sc = oracle.macko_spmv(W.n_cols, *enc, host(x[t]).view(np.uint16))
        bound = torch.from_numpy(sc) * ((W.n_cols / 32 + 76) * R.ADD)
        R.check(y[t], torch.from_numpy(yr), bound, f"token {t}")
        R.check(one, torch.from_numpy(yr), bound, f"vector {t}")


def test_strides_and_alignment():
    rows, cols, T = 90, 1000, 21
    w = _weight(rows, cols, "0.6", 4, 8)
    m = _matrix(w, rows, cols, 4)
    x0 = _x(T, cols, 4)
    ref, bound = R.spmm(w[4], x0, 1.0, 0.0, None, torch.float32)
    for extra, off in ((24, 0), (24, 8), (7, 0), (1, 1), (8, 3)):
        xb = torch.full((T, cols + extra + off), NAN, device="cuda").half()    # NaN around the rows is never read into a sum
        x = xb[:, off:off + cols]
        x.copy_(x0)
        yb = torch.full((T, rows + extra + off), -7.0, device="cuda")
        y = yb[:, off:off + rows]
        m.apply(x, y, workspace=m.workspace(T))
        R.check(y, ref, bound, f"{extra} {off}")
        assert (yb[:, :off] == -7).all() and (yb[:, off + rows:] == -7).all()
    with pytest.raises(S.SpmvError):                                           # needs a workspace
        S.macko_spmm(rows, cols, m.mrow_ptr, m.codes, m.vals, m.plan, 1.0, xb[:, 3:3 + cols], 0.0, y)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("cuts", [[0, 3, 3, 20, 90], [0, 0, 0, 0, 0], [5, 6, 70, 71, 80], [0, 90, 90, 90, 90], [0, 1, 2, 3, 4]])
def test_groups(cuts, i8):
    groups, rows, cols, T = 4, 72, 776, 90
    w = _weight(groups * rows, cols, "ragged", 4, 9, i8)
    m = _matrix(w, rows, cols, 4, groups)
    x = _x(T, cols, 2)
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    y0 = torch.randn(T, rows, device="cuda")
    y = y0.clone()
    m.apply(x, y, 1.0, 0.5, tok_offsets=off)
    ref, bound = R.f64(y0).clone(), torch.zeros(T, rows, dtype=torch.float64)
    for g in range(groups):
        a, b = cuts[g], cuts[g + 1]
        ref[a:b], bound[a:b] = R.spmm(w[4][g * rows:(g + 1) * rows], x[a:b], 1.0, 0.5, y0[a:b], torch.float32)
    R.check(y, ref, bound, str(cuts))


def test_offsets_outside_the_tokens_are_clamped():
    groups, rows, cols, T = 3, 16, 256, 10
    w = _weight(groups * rows, cols, "0.5", 4, 9)
    m = _matrix(w, rows, cols, 4, groups)
    x, y = _x(T, cols, 2), torch.zeros(T, rows, device="cuda")
    m.apply(x, y, tok_offsets=torch.tensor([-5, 4, 2, 1000], dtype=torch.int32, device="cuda"))
    # groups are rows 0..3, none and 2..9: rows 2 and 3 belong to two groups and may hold either's result
    for g, a, b in ((0, 0, 2), (2, 4, 10)):
        ref, bound = R.spmm(w[4][g * rows:(g + 1) * rows], x[a:b], 1.0, 0.0, None, torch.float32)
        R.check(y[a:b], ref, bound, "clamped")
    assert torch.isfinite(y).all()


def test_transpose_gives_the_gradient_in_x():
    """<dy, x W^T> is linear in x: its gradient dy W is the same call on the encoding of W^T."""
    rows, cols, T = 80, 520, 30
    w = _weight(rows, cols, "0.7", 4, 11)
    dense = w[4].numpy()
    t = dense.T
    rp = np.concatenate([[0], np.cumsum((t != 0).sum(1))]).astype(np.int32)
    ci = np.nonzero(t)[1].astype(np.int32)
    enc = S.macko_encode(cols, rows, rp, ci, t[t != 0].astype(np.float16).view(np.uint16))
    mt = _matrix((enc[0], enc[1], enc[2].view(np.float16), None, None), cols, rows, 4)
    dy = _x(T, rows, 3)
    dx = mt.apply(dy, torch.empty(T, cols, device="cuda"))
    ref, bound = R.spmm(torch.from_numpy(t.copy()), dy, 1.0, 0.0, None, torch.float32)
    R.check(dx, ref, bound, "dx")
    m = _matrix(w, rows, cols, 4)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, v = ((torch.randint(-8, 9, (T, cols), device="cuda", generator=g) / 8).half() for _ in range(2))
    run = lambda z: R.f64(m.apply(z, torch.empty(T, rows, device="cuda")))  # noqa: E731
    got = ((run(x + v) - run(x - v)) / 2 * R.f64(dy)).sum()
    want = (R.f64(dx) * R.f64(v)).sum()
    mag = (2 * torch.ones(T, cols, dtype=torch.float64) @ w[4].abs().t() * R.f64(dy).abs()).sum()
    assert abs(got - want) <= mag * 2 * (cols / 32 + 76) * R.ADD


def test_bad_token_stays_alone():
    rows, cols, T = 40, 700, 35
    w = _weight(rows, cols, "0.5", 4, 4)
    m = _matrix(w, rows, cols, 4)
    x = _x(T, cols, 6)
    ws = m.workspace(T)
    y0 = m.apply(x, torch.empty(T, rows, device="cuda"), workspace=ws).clone()
    x[4, 100], x[20, 699] = NAN, float("inf")
    y = m.apply(x, torch.empty(T, rows, device="cuda"), workspace=ws)
    keep = [t for t in range(T) if t not in (4, 20)]
    assert torch.equal(y[keep], y0[keep])


def test_graph_replays():
    rows, cols, T = 200, 1032, 40
    w = _weight(rows, cols, "0.7", 4, 4)
    m = _matrix(w, rows, cols, 4)
    buf = torch.zeros(T, cols + 1, device="cuda").half()
    for x in (torch.zeros(T, cols, device="cuda").half(), buf[:, 1:]):         # aligned, and packed first
        y, ws = torch.zeros(T, rows, device="cuda"), m.workspace(T)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.apply(x, y, workspace=ws)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.apply(x, y, workspace=ws)
        for i in range(3):
            x.copy_(_x(T, cols, 50 + i))
            y.fill_(NAN)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            want = m.apply(x, torch.empty_like(y), workspace=torch.empty_like(ws))
            assert torch.equal(y, want), i


def test_refusals_of_shapes():
    w = _weight(32, 64, "0.5", 4, 1)
    m = _matrix(w, 32, 64, 4)
    x, y = _x(4, 64, 1), torch.zeros(4, 32, device="cuda")
    for a, k, err in (((x[:, :63], y), {}, ValueError), ((x, y[:3]), {}, ValueError), ((x.float(), y), {}, TypeError),
                      ((x, y.bfloat16()), {}, TypeError), ((x, y.cpu()), {}, (TypeError, ValueError, AssertionError)),
                      ((x, y), dict(tok_offsets=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
                      ((x[:1].expand(4, 64), y), {}, ValueError)):
        with pytest.raises(err):
            m.apply(*a, **k)
    with pytest.raises(ValueError):
        S.MackoMatrix(31, 64, m.mrow_ptr, m.codes, m.vals)
    with pytest.raises(ValueError):
        S.macko_spmm(32, 64, m.mrow_ptr, m.codes, m.vals, m.plan[:8], 1.0, x, 0.0, y)
