"""The expert layer of 4-bit weights on the GPU against 64 bits: dropped and
repeated choices, idle experts, sizes, types, and replays."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
import quant_refs as Q  # noqa: E402

pytestmark = pytest.mark.gpu

F = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


class Layer:
    def __init__(self, experts, dim, inter, group, dt, zeros, seed):
        up = Q.weight(experts * 2 * inter, dim, group, F[dt], zeros, seed, scale=0.4 / dim ** 0.5)
        dn = Q.weight(experts * dim, inter, group, F[dt], zeros, seed + 1, scale=0.4 / inter ** 0.5)
        cuda = lambda w: [None if t is None else t.cuda() for t in w]  # noqa: E731
        self.gu = S.Q4Matrix(2 * inter, dim, *cuda(up), group=group, n_groups=experts)
        self.dn = S.Q4Matrix(dim, inter, *cuda(dn), group=group, n_groups=experts)
        self.up64 = Q.dense(*up, group, dim).view(experts, 2 * inter, dim)
        self.dn64 = Q.dense(*dn, group, inter).view(experts, dim, inter)
        self.dt, self.dim, self.inter, self.group = F[dt], dim, inter, group

    def __call__(self, keys, w, x, y=None):
        y = torch.full((x.shape[0], self.dim), float("nan"), device="cuda") if y is None else y
        ws = torch.empty(S.moe_workspace_size(keys.shape[0], keys.shape[1], self.dim, self.inter), dtype=torch.uint8, device="cuda")
        ws.fill_(255)
        return S.moe_apply(keys, w, self.gu, self.dn, x, y, ws)

    def check(self, keys, w, x, y, what=""):
        ref, bound = Q.moe(keys.cpu(), None if w is None else w.cpu(), self.up64, self.dn64, x, y.dtype, self.group)
        R.check(y, ref, bound, what)


def _batch(T, k, e, dim, dt, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    if kind == "mixed":
        keys = rng.integers(-1, e + 1, (T, k))               # some outside on either side, some twice
    elif kind == "one":
        keys = np.full((T, k), e - 1)
    elif kind == "none":
        keys = np.full((T, k), -1)
    else:
        keys = np.stack([rng.permutation(e)[:k] for _ in range(T)])
    x = torch.from_numpy(rng.standard_normal((T, dim)).astype(np.float32)).to(F[dt]).cuda()
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    return torch.from_numpy(keys.astype(np.int32)).cuda(), w, x


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,k,e", [(1, 2, 8), (5, 2, 3), (40, 3, 6)])
def test_types_and_groups(dt, group, zeros, T, k, e):
    m = Layer(e, 264, 200, group, dt, zeros, seed=group)
    keys, w, x = _batch(T, k, e, 264, dt, T)
    y = m(keys, w, x, torch.full((T, 264), float("nan"), device="cuda").to(F[dt] if T == 5 else torch.float32))
    m.check(keys, w, x, y)


@pytest.mark.parametrize("dim,inter", [(8, 1), (16, 7), (17, 128), (9, 2), (130, 129), (600, 520), (1000, 33)])
@pytest.mark.parametrize("T", [1, 4])
def test_sizes(dim, inter, T):
    m = Layer(4, dim, inter, 32, "bf16", True, seed=dim)
    keys, w, x = _batch(T, 2, 4, dim, "bf16", T, "distinct")
    m.check(keys, w, x, m(keys, w, x), f"{dim} {inter}")


@pytest.mark.parametrize("kind", ["mixed", "one", "none", "distinct"])
@pytest.mark.parametrize("T,k,e", [(1, 1, 1), (2, 8, 8), (16, 4, 64), (17, 1, 2), (64, 2, 5), (65, 2, 5), (256, 2, 4),
                                   (256, 16, 1000), (200, 20, 40), (1, 64, 1024)])
def test_choices(kind, T, k, e):
    m = Layer(e, 72, 40, 64, "f16", False, seed=e)
    keys, w, x = _batch(T, k, e, 72, "f16", T + k, kind)
    y = m(keys, w, x)
    m.check(keys, w, x, y, kind)
    if kind == "none":
        assert (y == 0).all()
    assert torch.equal(y, m(keys, w, x))                     # the same bits again


@pytest.mark.parametrize("group,zeros", [(128, False), (128, True), (32, True)])
@pytest.mark.parametrize("T,k,e", [(200, 4, 24), (250, 3, 40), (256, 4, 16), (90, 2, 24)])
def test_uneven_experts(T, k, e, group, zeros):
    """From no token to almost all of them: every number of turns and of tiles in a turn."""
    m = Layer(e, 300, 420, group, "f16", zeros, seed=e)
    keys, w, x = _batch(T, k, e, 300, "f16", T)
    g = torch.Generator().manual_seed(T)
    p = torch.pow(0.8, torch.arange(e - 1).double()).repeat(T, 1)
    keys = torch.multinomial(p, k, generator=g).to(torch.int32).to(keys.device)
    m.check(keys, w, x, m(keys, w, x))


def test_without_weights_and_strided():
    m = Layer(6, 136, 100, 128, "bf16", True, seed=3)
    keys, _, x = _batch(9, 2, 6, 136, "bf16", 4)
    wide, out = torch.full((9, 150), float("nan"), device="cuda").bfloat16(), torch.full((9, 141), 7.0, device="cuda").bfloat16()
    wide[:, 3:139] = x
    y = m(keys, None, wide[:, 3:139], out[:, 5:])
    m.check(keys, None, x, y)
    assert (out[:, :5] == 7.0).all()


def test_small_and_cancelling_hidden_values():
    """Down weights that cancel the large part of h leave what 16 bits of it would not hold."""
    dim, inter = 128, 128
    m = Layer(1, dim, inter, 128, "f16", False, seed=11)
    q = np.full((dim, inter), 8)
    q[:, 0], q[:, 1] = 15, 1                                 # y = 7 s (h0 - h1)
    s = torch.full((dim, 1), 0.25).half()
    m.dn = S.Q4Matrix(dim, inter, Q.pack(q).cuda(), s.cuda(), None, group=128)
    m.dn64 = Q.dense(Q.pack(q), s, None, 128, inter).view(1, dim, inter)
    w, s, _ = Q.weight(2 * inter, dim, 128, torch.float16, False, 12, scale=0.04)
    u = Q.unpack(w)
    u[1], u[inter + 1] = u[0], u[inter]
    s[1], s[inter + 1] = s[0], s[inter] * 1.001              # h1 is h0 but for a thousandth
    m.gu = S.Q4Matrix(2 * inter, dim, Q.pack(u).cuda(), s.cuda(), None, group=128)
    m.up64 = Q.dense(Q.pack(u), s, None, 128, dim).view(1, 2 * inter, dim)
    keys, w, x = _batch(8, 1, 1, dim, "f16", 2, "one")
    m.check(keys, w, x, m(keys, w, x))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_infinities_and_nan_stay_with_their_token(dt):
    m = Layer(3, 150, 90, 64, dt, False, seed=7)
    keys, w, x = _batch(20, 2, 3, 150, dt, 5, "distinct")
    x[4, 10], x[11, 149] = float("inf"), float("nan")
    y = m(keys, w, x)
    assert torch.isnan(y[11]).all() and not torch.isfinite(y[4]).any()
    keep = [t for t in range(20) if t not in (4, 11)]
    m.check(keys[keep], w[keep], x[keep], y[keep])


def test_large_hidden_values():
    """h near fp32's largest numbers is cut into parts without passing it."""
    dim = inter = 128
    m = Layer(1, dim, inter, 128, "bf16", False, seed=1)
    q = np.full((2 * inter, dim), 8)
    q[:, 0] = 15
    m.gu = S.Q4Matrix(2 * inter, dim, Q.pack(q).cuda(), torch.ones(2 * inter, 1, dtype=torch.bfloat16, device="cuda"), None)
    dn = np.full((dim, inter), 8)
    dn[:, 5] = 9
    m.dn = S.Q4Matrix(dim, inter, Q.pack(dn).cuda(), torch.full((dim, 1), 2.0 ** -20, dtype=torch.bfloat16, device="cuda"), None)
    x = torch.zeros(3, dim, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 2.6e18, 3.0e18, 1.0
    y = m(torch.zeros(3, 1, dtype=torch.int32, device="cuda"), None, x).cpu().double()
    xf = x.cpu().double()[:, 0] * 7
    ref = xf * torch.sigmoid(xf) * xf * 2.0 ** -20
    assert float(xf[0]) ** 2 < 3.4e38 < float(xf[1]) ** 2
    assert torch.isnan(y[1]).all()        # all of h is past fp32, and its other columns meet weights of 0: 0 * inf
    for t in (0, 2):
        assert ((y[t] - ref[t]).abs() <= ref[t].abs() * 2.0 ** -20).all()


def test_refusals():
    m = Layer(4, 72, 40, 64, "f16", False, seed=1)
    keys, w, x = _batch(5, 2, 4, 72, "f16", 1)
    y, ws = torch.empty(5, 72, device="cuda"), torch.empty(S.moe_workspace_size(5, 2, 72, 40), dtype=torch.uint8, device="cuda")
    ok = dict(keys=keys, weights=w, gate_up=m.gu, down=m.dn, x=x, y=y, workspace=ws)
    S.moe_apply(**ok)
    for name, bad in (("keys", keys.reshape(-1)), ("keys", keys[:4]), ("weights", w[:, :1]), ("x", x[:, :71]), ("y", y[:4]),
                      ("y", y[:, :71]), ("gate_up", m.dn), ("down", m.gu), ("workspace", ws[::2])):
        with pytest.raises(ValueError):
            S.moe_apply(**{**ok, name: bad})
    for name, bad in (("keys", keys.long()), ("weights", w.half()), ("x", x.bfloat16()), ("x", x.float()), ("y", y.bfloat16())):
        with pytest.raises(TypeError):
            S.moe_apply(**{**ok, name: bad})
    for bad in (None, ws[:-16]):
        with pytest.raises(S.SpmvError):
            S.moe_apply(**{**ok, "workspace": bad})
    other = Layer(4, 72, 40, 32, "f16", False, seed=1)
    with pytest.raises(ValueError):                          # another group size
        S.moe_apply(**{**ok, "down": other.dn})
    zeros = Layer(4, 72, 40, 64, "f16", True, seed=1)
    with pytest.raises(ValueError):                          # zero points in one of them
        S.moe_apply(**{**ok, "down": zeros.dn})


def test_captured_and_replayed():
    m = Layer(8, 256, 192, 64, "f16", True, seed=2)
    keys, w, x = _batch(24, 2, 8, 256, "f16", 1)
    y = torch.empty(24, 256, dtype=torch.float16, device="cuda")
    ws = torch.empty(S.moe_workspace_size(24, 2, 256, 192), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S.moe_apply(keys, w, m.gu, m.dn, x, y, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.moe_apply(keys, w, m.gu, m.dn, x, y, ws)
    for i in range(4):
        k2, w2, x2 = _batch(24, 2, 8, 256, "f16", 30 + i)
        keys.copy_(k2), w.copy_(w2), x.copy_(x2)
        y.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        m(*_batch(7, 2, 8, 256, "f16", 90 + i))
        torch.cuda.synchronize()
        assert torch.equal(y, m(keys, w, x, torch.empty_like(y))), i
