"""The 4-bit product of large weights with a decoding batch, whose tokens share x in
tiles of 16 to 64: types, groups, zero points, columns whole and split over workgroups,
a last block with fewer columns, against 64 bits in some of the rows."""
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
import quant_refs as Q  # noqa: E402

pytestmark = pytest.mark.gpu

F = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _run(rows, cols, tok, group, dt, zeros, ydt, alpha=1.0, beta=0.0, pad=0, large=1.0):
    """Every row is computed, 16 of each end and 32 between them are compared."""
    dt = F[dt]
    g = torch.Generator(device="cuda").manual_seed(rows + cols + tok)
    n = Q.blocks(cols) * 128
    codes = torch.randint(-2 ** 31, 2 ** 31, (rows, n // 8), device="cuda", generator=g).to(torch.int32)
    scales = ((torch.rand(rows, n // group, device="cuda", generator=g) + 0.25) * (0.05 / large ** 0.75)).to(dt)
    points = torch.randint(0, 16, scales.shape, device="cuda", generator=g).to(torch.uint8) if zeros else None
    m = S.Q4Matrix(rows, cols, codes, scales, points, group=group)
    x = torch.full((tok, cols + pad), float("nan"), dtype=dt, device="cuda")[:, pad:]
    x.copy_(torch.randn(tok, cols, device="cuda", generator=g).clamp_(-2.9, 2.9) * large)
    wide = torch.full((tok, rows + pad), float("nan"), dtype=dt if ydt == "x" else F[ydt], device="cuda")
    y = wide[:, pad:]
    if beta:
        y.copy_(torch.randn(tok, rows, device="cuda", generator=g))
    y_in = y.clone()
    ws = m.workspace(tok)
    ws.fill_(255)
    m.apply(x, y, alpha=alpha, beta=beta, workspace=ws)
    some = torch.cat([torch.arange(16), torch.arange(rows - 16, rows),
                      torch.randint(16, rows - 16, (32,), generator=torch.Generator().manual_seed(tok))])
    take = lambda t: t[some.cuda()].cpu()  # noqa: E731
    w = Q.dense(take(codes), take(scales), None if points is None else take(points), group, cols)
    ref, bound = Q.matmul(w, x, alpha, beta, y_in[:, some.cuda()], y.dtype, group)
    what = f"{rows}x{cols} tok {tok} group {group} {dt} zeros {zeros} y {ydt}"
    R.check(y[:, some.cuda()], ref, bound, what)
    assert not torch.isnan(y).any() and torch.isnan(wide[:, :pad]).all(), what
    first = y.clone()
    y.copy_(y_in)
    assert torch.equal(first, m.apply(x, y, alpha=alpha, beta=beta)), what


# 97 row tiles of 128: the columns are split over five workgroups, whose parts begin at odd blocks
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("tok", [5, 16, 17, 33, 48, 64])
def test_split(dt, group, zeros, tok):
    _run(12299, 12300, tok, group, dt, zeros, "f32" if tok % 2 else "x")


# more row tiles than workgroups on the card: a workgroup has all columns
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("tok", [7, 32, 47, 60])
def test_whole(dt, group, zeros, tok):
    _run(40001, 2500, tok, group, dt, zeros, "x" if tok % 2 else "f32")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols,tok", [(12299, 12300, 9), (12299, 12300, 30), (12299, 12300, 45), (40001, 2500, 21)])
@pytest.mark.parametrize("alpha,beta", [(-0.5, 1.0), (2.0, -0.25)])
def test_alpha_beta_and_strides(dt, rows, cols, tok, alpha, beta):
    _run(rows, cols, tok, 64, dt, True, "x" if alpha < 0 else "f32", alpha, beta, pad=3)


@pytest.mark.parametrize("rows,cols,tok", [(12299, 12300, 9), (12299, 12300, 30), (12299, 12300, 45), (40001, 2500, 21)])
def test_large_bf16(rows, cols, tok):
    """Numbers whose products with a code pass fp32's largest; the scale brings them back."""
    _run(rows, cols, tok, 64, "bf16", True, "f32", large=2.0 ** 126)


# 64 rows of a wave, columns whole, the last block, row tile and token tile in part
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols,tok", [(700, 850, 70), (700, 850, 200), (12299, 1020, 130), (129, 12300, 65)])
def test_wide_row_tiles(dt, rows, cols, tok):
    _run(rows, cols, tok, 128, dt, False, "f32" if tok % 2 else "x")


def test_captured_and_replayed():
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, cols, tok = 12299, 12300, 40
    m = S.Q4Matrix.quantize(torch.randn(rows, cols, device="cuda", generator=g).bfloat16(), group=64, zeros=True)
    x = torch.randn(tok, cols, device="cuda", generator=g).bfloat16()
    y, ws = torch.empty(tok, rows, device="cuda"), m.workspace(tok)
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
        x.copy_(torch.randn(tok, cols, device="cuda", generator=g))
        y.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        z = m.apply(x[:17], torch.empty(17, rows, device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(y, m.apply(x, torch.empty_like(y))), i
        assert torch.isfinite(z).all()
