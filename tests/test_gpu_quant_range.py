"""bf16 over its whole range in the 4-bit products and the expert layer: numbers whose
products with a code pass fp32's largest where the scale brings the result back, scales
as large, and results next to zero."""
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
import quant_refs as Q  # noqa: E402

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
TOP = torch.finfo(BF).max
# Tokens and columns of every form of the product: x in LDS, x per wave, tiles of shared x whole and split.
FORMS = [(1, 300), (3, 300), (5, 300), (20, 300), (33, 300), (64, 300), (70, 300), (70, 1100)]


def _weight(rows, cols, group, zeros, seed, scale):
    """Random codes; rows of the largest factors of either sign (15 and -15, or -8 and 7)."""
    n = Q.blocks(cols) * 128
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (rows, n), generator=g)
    z = torch.randint(0, 16, (rows, n // group), generator=g).to(torch.uint8) if zeros else None
    q[0], q[1] = 15, 0
    if zeros:
        z[0], z[1] = 0, 15
    s = ((torch.rand(rows, n // group, generator=g) + 0.25) * scale).to(BF)
    return Q.pack(q.numpy()), s, z


def _apply(w, rows, cols, group, x):
    m = S.Q4Matrix(rows, cols, *[None if t is None else t.cuda() for t in w], group=group)
    return m.apply(x.cuda(), torch.full((x.shape[0], rows), float("nan"), device="cuda"))


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("tok,cols", FORMS)
def test_large_x(tok, cols, group, zeros):
    rows = 40
    w = _weight(rows, cols, group, zeros, tok, 2.0 ** -20)
    g = torch.Generator().manual_seed(cols + tok)
    x = torch.randint(0, 2, (tok, cols), generator=g).double() * 2 - 1
    x = (x * TOP * torch.exp2(-20 * torch.rand(tok, cols, generator=g).double())).to(BF)
    x[0] = TOP
    ref, bound = Q.matmul(Q.dense(*w, group, cols), x, 1.0, 0.0, None, torch.float32, group)
    assert float(ref.abs().max()) < 1e38
    R.check(_apply(w, rows, cols, group, x), ref, bound, f"{tok} {cols} {group} {zeros}")


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("tok,cols", FORMS)
def test_large_scales(tok, cols, group, zeros):
    """Scales near fp32's largest number with an x that brings the result back."""
    rows = 40
    w = _weight(rows, cols, group, zeros, tok, 2.0 ** 127)
    x = (torch.randn(tok, cols, generator=torch.Generator().manual_seed(tok)).double() * 2.0 ** -100).to(BF)
    ref, bound = Q.matmul(Q.dense(*w, group, cols), x, 1.0, 0.0, None, torch.float32, group)
    R.check(_apply(w, rows, cols, group, x), ref, bound, f"{tok} {cols}")
    x = torch.full((tok, cols), 2.0 ** 10, dtype=BF)         # and where nothing does: an infinity of the sum's sign
    y = _apply(w, rows, cols, group, x).cpu()
    assert (y[:, 0] == float("inf")).all() and (y[:, 1] == float("-inf")).all()


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("tok,cols", FORMS)
@pytest.mark.parametrize("power", [-133, -126, -110])
def test_small_x(tok, cols, group, zeros, power):
    """From the smallest subnormal numbers on.  Sums are kept 2^11 times smaller than the
    result: where they are subnormal in fp32, adding a group rounds by 2^-150 of them, 2^-139
    of the result."""
    rows = 40
    w = _weight(rows, cols, group, zeros, tok, 1.0)
    g = torch.Generator().manual_seed(tok)
    x = (torch.randint(-127, 128, (tok, cols), generator=g).double() * 2.0 ** power).to(BF)
    ref, bound = Q.matmul(Q.dense(*w, group, cols), x, 1.0, 0.0, None, torch.float32, group)
    R.check(_apply(w, rows, cols, group, x), ref, bound + Q.blocks(cols) * (128 // group) * 2.0 ** -139, f"{tok} {cols}")


def _layer(experts, dim, inter, group, zeros, up, down):
    """up, down: (codes, scales, zero points) of the stacked rows."""
    gu = S.Q4Matrix(2 * inter, dim, up[0].cuda(), up[1].cuda(), None if up[2] is None else up[2].cuda(), group=group,
                    n_groups=experts)
    dn = S.Q4Matrix(dim, inter, down[0].cuda(), down[1].cuda(), None if down[2] is None else down[2].cuda(), group=group,
                    n_groups=experts)
    return gu, dn


def _experts(T, experts, gu, dn, x):
    keys = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(S.moe_workspace_size(T, 1, dn.n_rows, dn.n_cols), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    return keys.cpu(), S.moe_apply(keys, None, gu, dn, x.cuda(), torch.full((T, dn.n_rows), float("nan"), device="cuda"), ws)


# Tokens and experts of every form: down by ballots (parts in one operand and not), up per wave and in tiles, down in
# tiles with parts in one operand and one, two and three tiles at once, choices counted by the grid.
LAYERS = [(3, 4), (20, 4), (64, 4), (68, 100), (70, 8), (70, 4), (70, 1), (140, 1)]


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("T,experts", LAYERS)
def test_experts_with_large_hidden_values(T, experts, group, zeros):
    """Hidden values near fp32's largest, times factors of 15 (of 8 without zero points), 128 of a sign in a group."""
    dim, inter = 40, 200
    n, m = Q.blocks(dim) * 128, Q.blocks(inter) * 128
    q = torch.full((experts * 2 * inter, n), 8)
    q[:, 0] = 9                                              # gate and up are x's first column
    up = Q.pack(q.numpy()), torch.ones(q.shape[0], n // group, dtype=BF), \
        torch.full((q.shape[0], n // group), 8, dtype=torch.uint8) if zeros else None
    down = _weight(experts * dim, inter, group, zeros, T, 2.0 ** -24)
    gu, dn = _layer(experts, dim, inter, group, zeros, up, down)
    x = torch.zeros(T, dim, dtype=BF)
    x[:, 0] = (2.0 ** 63 * (0.5 + 0.9 * torch.rand(T, generator=torch.Generator().manual_seed(T)))).to(BF)
    x[0, 0] = 2.0 ** 63 * 1.984375                           # its square is 0.984 * 2^128
    keys, y = _experts(T, experts, gu, dn, x)
    ref, bound = Q.moe(keys, None, Q.dense(*up, group, dim).view(experts, 2 * inter, dim),
                       Q.dense(*down, group, inter).view(experts, dim, inter), x, torch.float32, group)
    assert float(ref.abs().max()) < 1e38
    R.check(y, ref, bound, f"{T} {experts}")


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("T,experts", LAYERS)
def test_experts_with_large_x(T, experts, group, zeros):
    dim, inter = 200, 40
    up = _weight(experts * 2 * inter, dim, group, zeros, T, 2.0 ** -120)
    down = _weight(experts * dim, inter, group, zeros, T + 1, 2.0 ** -6)
    gu, dn = _layer(experts, dim, inter, group, zeros, up, down)
    g = torch.Generator().manual_seed(T)
    x = (TOP * (2 * torch.rand(T, dim, generator=g).double() - 1)).to(BF)
    x[0] = TOP
    keys, y = _experts(T, experts, gu, dn, x)
    ref, bound = Q.moe(keys, None, Q.dense(*up, group, dim).view(experts, 2 * inter, dim),
                       Q.dense(*down, group, inter).view(experts, dim, inter), x, torch.float32, group)
    R.check(y, ref, bound, f"{T} {experts}")


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("tok,cols", FORMS)
def test_sums_that_alpha_brings_back(tok, cols, group, zeros):
    rows = 40
    w = _weight(rows, cols, group, zeros, tok, 2.0 ** -4)
    x = torch.full((tok, cols), TOP * 0.75, dtype=torch.float64).to(BF)
    m = S.Q4Matrix(rows, cols, *[None if t is None else t.cuda() for t in w], group=group)
    ref, bound = Q.matmul(Q.dense(*w, group, cols), x, 2.0 ** -11, 0.0, None, torch.float32, group)
    # of these rows the sum, before alpha, is past fp32's largest number, and less than 2^11 times it
    some = (ref.abs() * 2.0 ** 11 > 2.0 ** 128) & (ref.abs() < 2.0 ** 127)
    assert some[:, :2].all()
    y = m.apply(x.cuda(), torch.full((tok, rows), float("nan"), device="cuda"), alpha=2.0 ** -11).cpu().double()
    assert ((y - ref).abs() <= bound)[some].all()


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("T,experts", LAYERS)
def test_experts_whose_results_the_weights_bring_back(T, experts, group, zeros):
    dim, inter = 40, 200
    n, m = Q.blocks(dim) * 128, Q.blocks(inter) * 128
    q = torch.full((experts * 2 * inter, n), 8)
    q[:, 0] = 9
    up = Q.pack(q.numpy()), torch.ones(q.shape[0], n // group, dtype=BF), \
        torch.full((q.shape[0], n // group), 8, dtype=torch.uint8) if zeros else None
    q = torch.full((experts * dim, m), 9)                    # the sum of 200 hidden values
    down = Q.pack(q.numpy()), torch.ones(q.shape[0], m // group, dtype=BF), \
        torch.full((q.shape[0], m // group), 8, dtype=torch.uint8) if zeros else None
    gu, dn = _layer(experts, dim, inter, group, zeros, up, down)
    x = torch.zeros(T, dim, dtype=BF)
    x[:, 0] = (2.0 ** 63 * (0.5 + 0.5 * torch.rand(T, generator=torch.Generator().manual_seed(T)))).to(BF)
    keys = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), 2.0 ** -9, device="cuda")
    ws = torch.empty(S.moe_workspace_size(T, 1, dim, inter), dtype=torch.uint8, device="cuda")
    y = S.moe_apply(keys, w, gu, dn, x.cuda(), torch.full((T, dim), float("nan"), device="cuda"), ws)
    ref, bound = Q.moe(keys.cpu(), w.cpu(), Q.dense(*up, group, dim).view(experts, 2 * inter, dim),
                       Q.dense(*down, group, inter).view(experts, dim, inter), x, torch.float32, group)
    assert float(ref.min()) * 2.0 ** 9 > 2.0 ** 128
    R.check(y, ref, bound, f"{T} {experts}")
