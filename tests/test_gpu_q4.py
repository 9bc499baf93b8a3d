"""Products with 4-bit weights on the GPU against 64 bits, over sizes, groups,
types, strides and alignments; the codes of a dense weight against NumPy exactly."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
import quant_refs as Q  # noqa: E402

pytestmark = pytest.mark.gpu

F = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _matrix(rows, cols, group, dt, zeros, seed):
    w = Q.weight(rows, cols, group, F[dt], zeros, seed)
    return S.Q4Matrix(rows, cols, *[None if t is None else t.cuda() for t in w], group=group), Q.dense(*w, group, cols)


def _rows(n, width, dt, layout, gen, fill=None):
    """[n, width] of its own, in a wider buffer, or at an odd offset and stride."""
    extra, first = {"packed": (0, 0), "strided": (64, 8), "odd": (3, 1)}[layout]
    buf = torch.randn(n, width + extra, device="cuda", generator=gen)
    buf = (buf if fill is None else torch.full_like(buf, fill)).to(dt)
    return buf[:, first:first + width], buf


def _run(rows, cols, tok, group, dt, zeros, ydt, layout="packed", alpha=1.0, beta=0.0, seed=0):
    m, w = _matrix(rows, cols, group, dt, zeros, seed + rows + cols)
    gen = torch.Generator(device="cuda").manual_seed(seed + tok)
    x, _ = _rows(tok, cols, F[dt], layout, gen)
    y, buf = _rows(tok, rows, F[dt] if ydt == "x" else F[ydt], layout, gen, None if beta else float("nan"))
    y_in, before = y.clone(), buf.clone()
    m.apply(x, y, alpha=alpha, beta=beta)
    ref, bound = Q.matmul(w, x, alpha, beta, y_in, y.dtype, group)
    R.check(y, ref, bound, f"{rows}x{cols} tok {tok} group {group} {dt} zeros {zeros} y {ydt} {layout}")
    y.copy_(y_in)                                            # what lies between the rows is as it was
    assert torch.equal(torch.nan_to_num(buf.float(), nan=-7.0), torch.nan_to_num(before.float(), nan=-7.0))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("tok", [1, 3, 16, 17, 40, 64, 65, 130])
def test_tokens_groups_types(dt, group, zeros, tok):
    _run(77, 1160, tok, group, dt, zeros, "f32" if tok % 2 else "x", seed=group)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 33, 300])
@pytest.mark.parametrize("cols", [1, 7, 8, 31, 127, 128, 129, 511, 512, 513, 1000, 2560])
@pytest.mark.parametrize("tok", [1, 20])
def test_sizes(rows, cols, tok):
    _run(rows, cols, tok, 64 if cols % 2 else 32, "bf16" if rows % 2 else "f16", cols % 3 == 0, "f32")


@pytest.mark.parametrize("layout", ["packed", "strided", "odd"])
@pytest.mark.parametrize("alpha,beta", [(1.0, 0.0), (-0.5, 1.0), (2.0, -0.25), (0.0, 1.0)])
@pytest.mark.parametrize("tok", [1, 9, 50])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_strides_alpha_beta(layout, alpha, beta, tok, dt):
    _run(130, 645, tok, 128, dt, True, "x" if alpha < 0 else "f32", layout, alpha, beta)


@pytest.mark.parametrize("rows,cols,tok", [(2048, 4096, 1), (2048, 4096, 33), (1000, 12288, 5), (600, 2048, 513),
                                           (12288, 256, 16), (300, 300, 2000)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_larger(rows, cols, tok, dt):
    _run(rows, cols, tok, 128, dt, tok % 2 == 0, "f32")


def test_nothing_to_do_and_no_columns():
    m, _ = _matrix(40, 256, 64, "f16", True, 1)
    m.apply(torch.empty(0, 256, dtype=torch.float16, device="cuda"), torch.empty(0, 40, dtype=torch.float16, device="cuda"))
    codes = torch.empty(20, 0, dtype=torch.int32, device="cuda")
    scales = torch.empty(20, 0, dtype=torch.bfloat16, device="cuda")
    e = S.Q4Matrix(20, 0, codes, scales)
    x, y = torch.empty(3, 0, dtype=torch.bfloat16, device="cuda"), torch.full((3, 20), 2.0, device="cuda")
    assert (e.apply(x, y, beta=1.5) == 3.0).all()
    y.fill_(float("nan"))
    assert (e.apply(x, y) == 0.0).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("tok", [4, 30, 100])
@pytest.mark.parametrize("cols", [640, 700])
def test_infinities_and_nan_stay_in_their_row(dt, tok, cols):
    """What the definition gives in float64, sign of infinity and NaN included."""
    m, w = _matrix(90, cols, 64, dt, False, 5)
    x = torch.randn(tok, cols, generator=torch.Generator().manual_seed(1)).to(F[dt])
    x[1, 3], x[2, cols - 1] = float("inf"), float("nan")
    x[3, 3], x[3, 4] = float("inf"), float("-inf")
    y = torch.empty(tok, 90, device="cuda")
    m.apply(x.cuda(), y)
    got, ref = y.cpu().double(), x.double() @ w.t()
    for t in (1, 2, 3):
        assert torch.equal(torch.isnan(got[t]), torch.isnan(ref[t])), t
        some = ~torch.isnan(ref[t])
        assert torch.equal(got[t][some], ref[t][some]), t
    keep = [t for t in range(tok) if t not in (1, 2, 3)]
    ref, bound = Q.matmul(w, x[keep], 1.0, 0.0, None, torch.float32, 64)
    R.check(y[keep], ref, bound, "other tokens")


@pytest.mark.parametrize("tok", [1, 9, 80])
def test_subnormal_x(tok):
    """fp16's smallest numbers are multiplied as they are."""
    m, w = _matrix(50, 700, 128, "f16", True, 8)
    x = (torch.randint(-1023, 1024, (tok, 700)).double() * 2.0 ** -24).half()
    y = m.apply(x.cuda(), torch.empty(tok, 50, device="cuda"))
    ref, bound = Q.matmul(w, x, 1.0, 0.0, None, torch.float32, 128)
    R.check(y, ref, bound)


def test_refusals():
    m, _ = _matrix(40, 256, 64, "f16", True, 1)
    x, y = torch.zeros(3, 256, device="cuda").half(), torch.zeros(3, 40, device="cuda")
    for bad in (x.bfloat16(), x.float()):
        with pytest.raises(TypeError):
            m.apply(bad, y)
    for bx, by in ((x[:, :255], y), (x, y[:2]), (x, y[:, :39]), (x[0], y), (x.t(), y)):
        with pytest.raises(ValueError):
            m.apply(bx, by)
    with pytest.raises(TypeError):
        m.apply(x, y.bfloat16())
    with pytest.raises(TypeError):
        m.apply(x.cpu(), y)
    with pytest.raises(ValueError):
        S.q4_matmul(40, 256, m.tiles[:-16], 1.0, x, 0.0, y, group=64, with_zeros=True)
    stack = S.Q4Matrix.quantize(torch.randn(2, 20, 64, device="cuda"))
    with pytest.raises(ValueError):
        stack.apply(torch.zeros(1, 64, device="cuda").half(), torch.zeros(1, 20, device="cuda"))
    codes, scales = torch.zeros(40, 32, dtype=torch.int32, device="cuda"), torch.ones(40, 4, device="cuda").half()
    for c, s in ((codes[:-1], scales), (codes, scales[:-1]), (codes, scales.t())):
        with pytest.raises(ValueError):
            S.Q4Matrix(40, 256, c, s, group=64)
    with pytest.raises(TypeError):
        S.Q4Matrix(40, 256, codes, scales.float(), group=64)
    with pytest.raises(ValueError):
        S.Q4Matrix(40, 256, codes, scales, group=48)
    big = S.Q4Matrix.quantize(torch.randn(2048, 12288, device="cuda").half())
    with pytest.raises(S.SpmvError):                         # the workspace of one token for 64
        big.apply(torch.zeros(64, 12288, device="cuda").half(), torch.zeros(64, 2048, device="cuda"), workspace=big.workspace(1))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("tok", [1, 16, 70])
def test_zero_weights_give_exact_zeros(dt, tok):
    """Codes equal to the zero point, whatever the scale: no residue of large products that cancel."""
    rows, cols, group = 48, 1100, 32
    n = Q.blocks(cols) * 128
    z = torch.randint(0, 16, (rows, n // group)).to(torch.uint8)
    q = torch.repeat_interleave(z, group, 1)
    s = torch.full(z.shape, 3.0, dtype=F[dt])
    m = S.Q4Matrix(rows, cols, Q.pack(q.numpy()).cuda(), s.cuda(), z.cuda(), group=group)
    x = (torch.randn(tok, cols, device="cuda") * 1e4).to(F[dt])
    assert (m.apply(x, torch.empty(tok, rows, device="cuda")) == 0).all()


@pytest.mark.parametrize("tok", [1, 16, 17, 64, 200])
def test_bits_repeat_and_do_not_depend_on_the_workspace(tok):
    m, _ = _matrix(520, 3000, 128, "bf16", True, 2)
    x = torch.randn(tok, 3000, device="cuda").to(torch.bfloat16)
    first = m.apply(x, torch.empty(tok, 520, device="cuda"))
    for n in (tok, tok + 1, 4 * tok, 1000):
        ws = m.workspace(n)
        ws.fill_(255)
        assert torch.equal(first, m.apply(x, torch.empty(tok, 520, device="cuda"), workspace=ws)), n


@pytest.mark.parametrize("src", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize(src, dt, group, zeros):
    rows, cols = 37, 300
    rng = np.random.default_rng(group)
    w = (rng.standard_normal((rows, cols)) * 0.1).astype(np.float32)
    w[3] = 0.0                                               # a row of zeros
    w[4, :200] = np.abs(w[4, :200])                          # groups of one sign
    w[5, :200] = -np.abs(w[5, :200])
    w[6] *= 1e-9                                             # scales that vanish in fp16
    if src != "f16":
        w[7] *= 1e8                                          # scales that do not fit fp16
    w[8, 130] = 5.0
    t = torch.from_numpy(w).to(F[src])
    wide = torch.full((rows, cols + 5), float("nan")).to(F[src])
    wide[:, 2:2 + cols] = t
    n = Q.blocks(cols) * 128
    codes = torch.empty(rows, n // 8, dtype=torch.int32, device="cuda")
    scales = torch.empty(rows, n // group, dtype=F[dt], device="cuda")
    points = torch.empty(rows, n // group, dtype=torch.uint8, device="cuda") if zeros else None
    S.q4_quantize(wide.cuda()[:, 2:2 + cols], codes, scales, points, group)
    full = np.zeros((rows, n), np.float32)
    full[:, :cols] = t.float().numpy()
    g = full.reshape(rows, n // group, group)
    hi, lo = np.maximum(g.max(2), 0), np.minimum(g.min(2), 0)
    f = np.float32
    want = hi / f(15) - lo / f(15) if zeros else np.maximum(hi, -lo) / f(7)
    s = torch.from_numpy(np.minimum(want, f(torch.finfo(F[dt]).max))).to(F[dt])
    assert torch.equal(scales.cpu(), s)
    sf = s.float().numpy()
    safe = np.where(sf > 0, sf, f(1))
    z = np.where(sf > 0, np.minimum(np.rint(-lo / safe), f(15)), f(0)) if zeros else np.full_like(sf, 8)
    if zeros:
        assert np.array_equal(points.cpu().numpy(), z.astype(np.uint8))
    q = np.where(sf[:, :, None] > 0, np.clip(np.rint(g / safe[:, :, None]) + z[:, :, None], 0, 15), z[:, :, None])
    assert np.array_equal(Q.unpack(codes), q.reshape(rows, n).astype(np.int64))


def test_quantize_of_a_strided_stack_on_another_stream():
    w = torch.randn(3, 20, 200, device="cuda").half()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    m, ref = S.Q4Matrix.quantize(w[:, :, 30:190], stream=side), S.Q4Matrix.quantize(w[:, :, 30:190].contiguous())
    torch.cuda.synchronize()
    assert (m.n_groups, m.n_rows, m.n_cols) == (3, 20, 160) and torch.equal(m.tiles, ref.tiles)
    with pytest.raises(ValueError):
        S.Q4Matrix.quantize(w[0, 0])


def test_quantized_weight_is_near_the_weight():
    """Half a step of the scale per weight (symmetric: the scale is at most max / 7 rounded)."""
    w = torch.randn(64, 500, device="cuda")
    m = S.Q4Matrix.quantize(w, group=32, dtype=torch.float16)
    x = torch.eye(500, device="cuda").half()                 # the weight's columns
    d = R.f64(m.apply(x, torch.empty(500, 64, device="cuda"))).t()
    top = R.f64(w).abs()
    top = torch.nn.functional.pad(top, (0, 12)).view(64, 16, 32).amax(2)
    step = torch.repeat_interleave(top / 7, 32, 1)[:, :500]
    assert ((d - R.f64(w)).abs() <= step * (0.5 + 8 * 2.0 ** -11)).all()
    assert S.Q4Matrix.quantize(torch.randn(3, 20, 40, device="cuda").bfloat16(), zeros=True).n_groups == 3


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,cols,group", [(1, 1, 128), (16, 128, 64), (35, 300, 32), (48, 129, 128)])
def test_tiles(rows, cols, group, zeros):
    """The records word for word; scales of groups past the last column are zeros."""
    w, s, z = Q.weight(rows, cols, group, torch.float16, zeros, rows)
    m = S.Q4Matrix(rows, cols, w.cuda(), s.cuda(), None if z is None else z.cuda(), group=group)
    nb, gb = Q.blocks(cols), 128 // group
    rec = m.tiles.cpu().numpy().reshape(-1, 1024 + gb * (48 if zeros else 32))
    s = s.clone()
    s[:, (cols + group - 1) // group:] = 0
    pad = lambda t: np.pad(t.numpy(), ((0, -rows % 16), (0, 0)))  # noqa: E731
    for i in range((rows + 15) // 16):
        for b in range(nb):
            r = rec[i * nb + b]
            codes = pad(w)[16 * i:16 * i + 16, 16 * b:16 * b + 16].reshape(16, 4, 4).transpose(1, 0, 2)
            assert np.array_equal(r[:1024].view(np.int32).reshape(4, 16, 4), codes)
            sc = pad(s)[16 * i:16 * i + 16, gb * b:gb * b + gb]
            assert np.array_equal(r[1024:1024 + 32 * gb].view(np.float16).reshape(16, gb), sc)
            if zeros:
                assert np.array_equal(r[1024 + 32 * gb:].reshape(16, gb), pad(z)[16 * i:16 * i + 16, gb * b:gb * b + gb])


@pytest.mark.parametrize("tok", [1, 12, 300])
@pytest.mark.parametrize("cols,group", [(300, 32), (129, 64)])
def test_scales_past_the_last_column_are_not_used(tok, cols, group):
    w, s, z = Q.weight(40, cols, group, torch.float16, True, 2)
    x = torch.randn(tok, cols, generator=torch.Generator().manual_seed(3)).half()
    ref, bound = Q.matmul(Q.dense(w, s, z, group, cols), x, 1.0, 0.0, None, torch.float32, group)
    s[:, (cols + group - 1) // group:] = float("nan")
    m = S.Q4Matrix(40, cols, w.cuda(), s.cuda(), z.cuda(), group=group)
    R.check(m.apply(x.cuda(), torch.empty(tok, 40, device="cuda")), ref, bound)


@pytest.mark.parametrize("tok", [1, 12, 40, 300])
def test_captured_and_replayed(tok):
    m, _ = _matrix(700, 2100, 64, "f16", True, 9)
    other, _ = _matrix(256, 2100, 32, "f16", False, 10)
    x = torch.randn(tok, 2100, device="cuda").half()
    y, ws = torch.empty(tok, 700, device="cuda"), m.workspace(tok)
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
        x.copy_(torch.randn(tok, 2100, device="cuda"))
        y.fill_(float("nan"))
        graph.replay()
        z = other.apply(x, torch.empty(tok, 256, device="cuda"))
        torch.cuda.synchronize()
        assert torch.isfinite(z).all()
        assert torch.equal(y, m.apply(x, torch.empty_like(y))), i


def test_other_stream_and_workspace_per_call():
    m, w = _matrix(512, 1024, 128, "f16", False, 3)
    x = torch.randn(20, 1024, device="cuda").half()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    ys = [torch.empty(20, 512, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for s, y in zip(streams, ys):
        m.apply(x, y, stream=s)
    torch.cuda.synchronize()
    ref, bound = Q.matmul(w, x, 1.0, 0.0, None, torch.float32, 128)
    for y in ys:
        R.check(y, ref, bound, "stream")
