"""The expert layer with more than 64 choices and no more choices than experts (each
choice's workgroup looks whether an earlier one has its expert), and hidden values to
their 24th bit in every form of the down product."""
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
import quant_refs as Q  # noqa: E402
from test_gpu_moe import Layer, _batch  # noqa: E402

@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["mixed", "one", "none", "distinct"])
@pytest.mark.parametrize("T,k,e", [(16, 8, 256), (40, 4, 300), (100, 10, 1000), (65, 1, 65), (256, 4, 1024)])
def test_more_than_64_choices_and_as_many_experts(kind, T, k, e):
    m = Layer(e, 72, 40, 64, "f16", False, seed=e)
    keys, w, x = _batch(T, k, e, 72, "f16", T + k, kind)
    y = m(keys, w, x)
    m.check(keys, w, x, y, kind)
    if kind == "none":
        assert (y == 0).all()
    assert torch.equal(y, m(keys, w, x))


@pytest.mark.gpu
@pytest.mark.parametrize("group,zeros,dt", [(32, True, "bf16"), (64, False, "f16"), (128, True, "f16"), (128, False, "bf16")])
@pytest.mark.parametrize("kind", ["mixed", "one"])
def test_more_than_64_choices_of_wider_layers(kind, group, zeros, dt):
    m = Layer(72, 300, 260, group, dt, zeros, seed=group)
    keys, w, x = _batch(24, 3, 72, 300, dt, 5, kind)
    y = m(keys, w, x, torch.full((24, 300), float("nan"), device="cuda").to(x.dtype))
    m.check(keys, w, x, y, kind)


DIM, INTER, LARGE = 72, 40, 2.0 ** 18


def _nearly_equal_hidden_values(T, dtype):
    """(x, y, bound) of a layer whose every output is 7 (h1 - h0), h0 = 2^18 silu(g) and h1 = (2^18 + d) silu(g), with d
    from 1 to 128.  g, 2^18 and d are exact.  Both hidden values have the same silu, and a product rounded by half a
    step, 2^-24 of 2^18 silu(g); their 6 products with 7 and -7 pass at most 6 additions of a whole step, 2^-23 of
    7 * 2^18 silu(g); what else is added is zeros."""
    g = torch.Generator().manual_seed(T)
    x = torch.zeros(T, DIM)
    x[:, 0] = 0.5 + 2.5 * torch.rand(T, generator=g)
    x[:, 32] = 8.0
    x[:, 64] = torch.exp2(torch.arange(T) % 8).float()
    x = x.to(dtype)
    silu, d = x[:, 0].double() * torch.sigmoid(x[:, 0].double()), x[:, 64].double()
    y = 7 * d * silu
    # the silu's own few roundings are the same in both
    bound = 7 * silu * LARGE * (2 * 2.0 ** -24 + 6 * 2.0 ** -23) + y * 16 * 2.0 ** -24
    return x, y, bound


def test_the_bound_tells_hidden_values_of_fewer_bits():
    x, y, bound = _nearly_equal_hidden_values(64, torch.float16)
    g = x[:, 0].float()
    silu = g / (1.0 + torch.exp(-g))
    h0, h1 = silu * LARGE, silu * (LARGE + x[:, 64].float())
    for bits, fits in ((24, True), (16, False), (19, False)):
        cut = lambda h: (h.view(torch.int32) & -(1 << (24 - bits))).view(torch.float32).double()  # noqa: B023, E731
        assert bool(((7 * (cut(h1) - cut(h0)) - y).abs() <= bound).all()) == fits, bits


# Tokens and experts of every form of the down product: parts in one operand (up to 5 tokens), one by one, in tiles
# (one, two and three of them), choices counted by the grid.
@pytest.mark.gpu
@pytest.mark.parametrize("T,experts", [(4, 2), (20, 2), (64, 2), (68, 100), (70, 8), (70, 4), (70, 1), (140, 1)])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_all_bits_of_the_hidden_values(T, experts, group, zeros, dt):
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16}[dt]
    x, ref, bound = _nearly_equal_hidden_values(T, dtype)
    q = torch.full((experts * 2 * INTER, 128), 8)
    s = torch.ones(q.shape[0], 128 // group)
    q[:2, 0] = 9                                             # gate rows 0 and 1: g
    q[INTER:INTER + 2, 32] = 9                               # up rows 0 and 1: 2^18, and d in the second
    q[INTER + 1, 64] = 9
    if group == 32:                                          # a group of its own for 2^18, or x as large
        s[INTER:INTER + 2, 1] = LARGE / 8.0
    else:
        x = x.clone()
        s[INTER:INTER + 2] = 2.0 ** 4
        x[:, 32], x[:, 64] = LARGE / 2 ** 4, x[:, 64] / 2 ** 4
    point = lambda t: torch.full(t.shape, 8, dtype=torch.uint8, device="cuda") if zeros else None  # noqa: E731
    gu = S.Q4Matrix(2 * INTER, DIM, Q.pack(q.numpy()).cuda(), s.to(dtype).cuda(), point(s), group=group, n_groups=experts)
    q = torch.full((experts * DIM, 128), 8)
    s = torch.ones(q.shape[0], 128 // group)
    q[:, 0], q[:, 1] = 1, 15
    dn = S.Q4Matrix(DIM, INTER, Q.pack(q.numpy()).cuda(), s.to(dtype).cuda(), point(s), group=group, n_groups=experts)
    keys = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(S.moe_workspace_size(T, 1, DIM, INTER), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    y = S.moe_apply(keys, None, gu, dn, x.cuda(), torch.full((T, DIM), float("nan"), device="cuda"), ws)
    R.check(y, ref[:, None].expand(T, DIM), bound[:, None].expand(T, DIM), f"{T} {experts}")
