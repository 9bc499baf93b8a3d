"""Low-rank adapters on the GPU against 64 bits: mixed ranks, tokens without
an adapter, odd widths and strides, both types, in place and not; the
gradients against the formula and against differences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402

pytestmark = pytest.mark.gpu

F = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


def _make(T, K, N, n, r, dt, seed, ranks="mixed", keys="mixed"):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if keys == "mixed":
        ks = rng.integers(-1, n + 1, T)
    elif keys == "one":
        ks = np.full(T, n // 2)
    elif keys == "none":
        ks = np.full(T, -1)
    else:
        ks = rng.integers(0, n, T)
    rk = {"mixed": rng.integers(-1, r + 3, n), "full": np.full(n, r), "zero": np.zeros(n, int)}[ranks]
    A = (torch.randn(n, r, K, device="cuda", generator=g) / K ** 0.5).to(F[dt])
    B = torch.randn(n, r, N, device="cuda", generator=g).to(F[dt])
    used = np.clip(rk, 0, r)
    for a in range(n):                        # what lies past a rank is never used
        A[a, used[a]:] = NAN
        B[a, used[a]:] = NAN
    x = torch.randn(T, K, device="cuda", generator=g).to(F[dt])
    scale = torch.rand(n, device="cuda", generator=g) * 3 - 1
    plan = S.RoutePlan(T, 1, n).build(torch.from_numpy(ks.astype(np.int32)).cuda())
    ws = torch.full((S.lora_workspace_size(T, r),), 255, dtype=torch.uint8, device="cuda")   # NaN
    return dict(keys=ks, ranks=used.tolist(), ranks_t=torch.from_numpy(rk.astype(np.int32)).cuda(), scale=scale,
                A=A, B=B, x=x, plan=plan, ws=ws)


def _clean(t, ranks):
    t = t.clone()
    for a, r in enumerate(ranks):
        t[a, r:] = 0
    return t


def _apply(s, x, y_in, y, A=None, B=None):
    p = s["plan"]
    out = S.lora_apply(s["ranks_t"], s["scale"], s["A"] if A is None else A, s["B"] if B is None else B, p.order,
                       p.offsets, p.tiles, x, y_in, y, s["ws"])
    torch.cuda.synchronize()
    return out


def _bits(dt, ydt):
    return 22 if dt == "f16" else (24 if ydt == torch.float32 else 16)


SHAPES = [(1, 64, 64, 1, 1), (1, 4096, 512, 4, 16), (3, 8, 8, 2, 8), (17, 1000, 1504, 3, 8), (40, 136, 648, 5, 24),
          (61, 2048, 1024, 40, 64), (200, 33, 77, 3, 5), (150, 515, 130, 2, 33), (70, 256, 264, 2, 128),
          (33, 264, 1032, 9, 100), (16, 64, 1, 2, 4), (31, 1, 64, 2, 4), (700, 1032, 520, 4, 16), (600, 200, 1048, 2, 64),
          (520, 129, 130, 1, 100), (513, 4096, 64, 8, 24), (45, 9, 131, 2, 8), (45, 7, 515, 2, 8), (45, 515, 7, 2, 8),
          (45, 1031, 129, 2, 20), (40, 8, 8, 2, 3)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("y32", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_apply(shape, dt, y32):
    T, K, N, n, r = shape
    s = _make(T, K, N, n, r, dt, seed=T + K)
    ydt = torch.float32 if y32 else F[dt]
    base = torch.randn(T, N, device="cuda").to(ydt)
    sc = R.f64(s["scale"]).tolist()
    args = (s["keys"], s["ranks"], sc, _clean(s["A"], s["ranks"]), _clean(s["B"], s["ranks"]), s["x"])
    y = torch.full_like(base, NAN)
    assert _apply(s, s["x"], base, y) is y
    ref, bound = R.lora(*args, base, _bits(dt, ydt), ydt)
    R.check(y, ref, bound, f"lora {shape} {dt}")
    again = base.clone()                       # in place: the same bits
    _apply(s, s["x"], again, again)
    assert torch.equal(again, y)
    y.fill_(NAN)
    _apply(s, s["x"], None, y)
    ref, bound = R.lora(*args, None, _bits(dt, ydt), ydt)
    R.check(y, ref, bound, f"lora delta {shape} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("keys", ["one", "none", "all"])
def test_apply_groups(keys, dt):
    s = _make(90, 512, 520, 6, 16, dt, seed=3, ranks="full", keys=keys)
    base = torch.randn(90, 520, device="cuda")
    y = torch.full_like(base, NAN)
    _apply(s, s["x"], base, y)
    ref, bound = R.lora(s["keys"], s["ranks"], R.f64(s["scale"]).tolist(), s["A"], s["B"], s["x"], base, _bits(dt, base.dtype),
                        base.dtype)
    R.check(y, ref, bound, keys)
    if keys == "none":
        assert torch.equal(y, base)


def test_default_rank_and_scale():
    s = _make(20, 128, 128, 3, 8, "f16", seed=8, ranks="full")
    s["ranks_t"] = None
    one, s["scale"] = s["scale"], None
    y = torch.empty(20, 128, device="cuda")
    _apply(s, s["x"], None, y)
    ref, bound = R.lora(s["keys"], s["ranks"], [1.0] * 3, s["A"], s["B"], s["x"], None, 22, y.dtype)
    R.check(y, ref, bound, "defaults")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_strides_and_alignment(dt):
    T, K, N = 37, 264, 392
    s = _make(T, K, N, 3, 16, dt, seed=4)
    sc = R.f64(s["scale"]).tolist()
    A, B = _clean(s["A"], s["ranks"]), _clean(s["B"], s["ranks"])
    for pad, off in ((64, 8), (5, 3), (1, 1)):
        xb = torch.full((T, K + pad + off), NAN, device="cuda").to(F[dt])
        x = xb[:, off:off + K]
        x.copy_(s["x"])
        yb = torch.full((T, N + pad + off), -5.0, device="cuda").to(F[dt])
        y = yb[:, off:off + N]
        base = torch.randn(T, N, device="cuda").to(F[dt])
        _apply(s, x, base, y)
        ref, bound = R.lora(s["keys"], s["ranks"], sc, A, B, x, base, 16, F[dt])
        R.check(y, ref, bound, f"strides {pad} {off}")
        assert (yb[:, :off] == -5).all() and (yb[:, off + N:] == -5).all()


def test_fp16_range_of_the_rank_vector():
    """A x past fp16's largest value, or far below its smallest, in different
    tokens of one tile."""
    T, K, N, r = 16, 512, 256, 16
    s = _make(T, K, N, 1, r, "f16", seed=5, ranks="full", keys="one")
    s["A"] = torch.randn(1, r, K, device="cuda").half()
    s["x"] *= torch.tensor([[10.0 ** (3 - t // 2)] for t in range(T)], device="cuda").half()
    s["B"] = (torch.randn(1, r, N, device="cuda") * 1e-3).half()
    s["scale"].fill_(1.0)
    y = torch.empty(T, N, device="cuda")
    _apply(s, s["x"], None, y)
    ref, bound = R.lora(s["keys"], [r], [1.0], s["A"], s["B"], s["x"], None, 22, y.dtype)
    assert torch.isfinite(y).all()
    R.check(y, ref, bound, "range")


def test_bad_token_stays_alone():
    s = _make(20, 256, 256, 1, 8, "bf16", seed=6, ranks="full", keys="one")
    y0 = torch.empty(20, 256, device="cuda")
    _apply(s, s["x"], None, y0)
    x = s["x"].clone()
    x[3, 5], x[7, 0] = NAN, float("inf")
    y = torch.empty_like(y0)
    _apply(s, x, None, y)
    keep = [t for t in range(20) if t not in (3, 7)]
    assert torch.equal(y[keep], y0[keep])
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[7]).any()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 64, 64, 1, 1), (300, 1000, 1504, 3, 8), (500, 136, 520, 4, 24), (77, 33, 70, 2, 5),
                                   (260, 512, 128, 1, 64), (90, 128, 264, 3, 128), (600, 64, 64, 20, 16),
                                   (2100, 1040, 1096, 2, 32), (1500, 72, 64, 3, 48), (700, 2560, 2056, 1, 16), (200, 1031, 515, 2, 16), (80, 9, 7, 2, 4),
                                   (600, 517, 135, 2, 32), (8200, 136, 72, 5, 32),
                                   (8199, 7, 265, 3, 20), (16390, 72, 40, 9, 12), (300, 33, 135, 70, 24),
                                   (600, 1032, 520, 20, 48), (130, 5, 9, 100, 100), (513, 264, 136, 50, 16)])
def test_grad(shape, dt):
    T, K, N, n, r = shape
    s = _make(T, K, N, n, r, dt, seed=T)
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = (torch.randn(T, N, device="cuda", generator=g) * 1e-3).to(F[dt])
    p = s["plan"]
    dA, dB = torch.full((n, r, K), NAN, device="cuda"), torch.full((n, r, N), NAN, device="cuda")
    S.lora_grad(s["ranks_t"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"], dy, dA, dB, s["ws"])
    torch.cuda.synchronize()
    sc = R.f64(s["scale"]).tolist()
    A, B = _clean(s["A"], s["ranks"]), _clean(s["B"], s["ranks"])
    ra, ba, rb, bb = R.lora_grad(s["keys"], s["ranks"], sc, A, B, s["x"], dy)
    R.check(dA, ra, ba, f"dA {shape} {dt}")
    R.check(dB, rb, bb, f"dB {shape} {dt}")
    again = (torch.empty_like(dA), torch.empty_like(dB))
    S.lora_grad(s["ranks_t"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"], dy, *again, s["ws"])
    assert torch.equal(again[0], dA) and torch.equal(again[1], dB)
    # the gradient in x: the same product with A and B exchanged
    dx = torch.full((T, K), NAN, device="cuda")
    _apply(s, dy, None, dx, A=s["B"], B=s["A"])
    ref, bound = R.lora(s["keys"], s["ranks"], sc, B, A, dy, None, _bits(dt, dx.dtype), dx.dtype)
    R.check(dx, ref, bound, f"dx {shape} {dt}")


def test_grad_of_tiny_and_large_tokens_together():
    """fp16: tokens whose rank vectors differ by 2^40 share one adapter."""
    T, K, N, r = 96, 256, 128, 8
    s = _make(T, K, N, 1, r, "f16", seed=21, ranks="full", keys="one")
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn(T, N, device="cuda", generator=g)
    dy[::2] *= 2.0 ** -20
    dy[32:48] *= 2.0 ** -14
    dy[48:64] *= 2.0 ** 8
    dy = dy.half()
    dA, dB = torch.empty(1, r, K, device="cuda"), torch.empty(1, r, N, device="cuda")
    p = s["plan"]
    S.lora_grad(s["ranks_t"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"], dy, dA, dB, s["ws"])
    ra, ba, rb, bb = R.lora_grad(s["keys"], [r], R.f64(s["scale"]).tolist(), s["A"], s["B"], s["x"], dy)
    R.check(dA, ra, ba, "dA")
    R.check(dB, rb, bb, "dB")


def test_grad_without_tokens():
    s = _make(0, 64, 72, 3, 8, "f16", seed=1)
    dA, dB = torch.full((3, 8, 64), NAN, device="cuda"), torch.full((3, 8, 72), NAN, device="cuda")
    p = s["plan"]
    S.lora_grad(s["ranks_t"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"],
                torch.zeros(0, 72, device="cuda").half(), dA, dB, s["ws"])
    assert (dA == 0).all() and (dB == 0).all()


def test_grad_is_the_difference_quotient():
    """<dy, y> is linear in A, in B and in x, so central differences with
    steps that the types hold exactly give the gradients up to y's rounding."""
    T, K, N, n, r = 50, 64, 96, 3, 8
    s = _make(T, K, N, n, r, "f16", seed=12, ranks="full", keys="all")
    g = torch.Generator(device="cuda").manual_seed(2)
    q = lambda *sh: (torch.randint(-8, 9, sh, device="cuda", generator=g) / 8).half()  # noqa: E731
    A, B, x, dy = q(n, r, K), q(n, r, N), q(T, K), q(T, N)
    s["scale"] = torch.tensor([1.0, 0.5, -2.0], device="cuda")
    p = s["plan"]
    dA, dB = torch.empty(n, r, K, device="cuda"), torch.empty(n, r, N, device="cuda")
    S.lora_grad(s["ranks_t"], s["scale"], A, B, p.order, p.offsets, p.tiles, x, dy, dA, dB, s["ws"])
    dx = _apply(s, dy, None, torch.empty(T, K, device="cuda"), A=B, B=A)
    run = lambda x, A, B: R.f64(_apply(s, x, None, torch.empty(T, N, device="cuda"), A=A, B=B))  # noqa: E731
    for name, grad, args in (("A", dA, lambda v: (x, A + v, B)), ("B", dB, lambda v: (x, A, B + v)),
                             ("x", dx, lambda v: (x + v, A, B))):
        v = q(*grad.shape)
        got = ((run(*args(v)) - run(*args(-v))) / 2 * R.f64(dy)).sum()
        want = (R.f64(grad) * R.f64(v)).sum()
        # y: K products of at most 2, r of them times 2, scale 2; every rounding at most (K / 32 + 3 r + 100) steps
        size = T * N * (K * 2 * r * 2 * 2)
        assert abs(got - want) <= size * ((K / 32 + 3 * r + 100) * R.ADD + 2.0 ** -22), name


def test_graph_replays_share_nothing_but_inputs():
    """Two captured graphs with workspaces of their own, replayed in turn with eager work between."""
    s = _make(64, 512, 768, 5, 16, "bf16", seed=9, ranks="full")
    base = torch.randn(64, 768, device="cuda")
    p, ws2 = s["plan"], s["ws"].clone()
    ys = [torch.empty_like(base), torch.empty_like(base)]

    def run(y, ws):
        S.lora_apply(s["ranks_t"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"], base, y, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(ys[0], s["ws"])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for y, ws in zip(ys, (s["ws"], ws2)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run(y, ws)
        graphs.append(gr)
    for i in range(3):
        s["x"].copy_(torch.randn(64, 512, device="cuda"))
        base.copy_(torch.randn(64, 768, device="cuda"))
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(base)
        run(want, torch.empty_like(s["ws"]))
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want) and torch.equal(ys[1], want)


def test_two_streams_at_once():
    s = _make(100, 1024, 1024, 4, 32, "f16", seed=10, ranks="full")
    base = torch.randn(100, 1024, device="cuda")
    p = s["plan"]
    want = _apply(s, s["x"], base, torch.empty_like(base))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for st in streams:
        y, ws = torch.empty_like(base), torch.empty_like(s["ws"])
        torch.cuda.synchronize()
        for _ in range(5):
            S.lora_apply(s["ranks_t"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"], base, y, ws, stream=st)
        outs.append((y, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y, _ in outs)


def test_a_plan_that_was_never_built_reads_and_writes_inside():
    """Any contents of the plan arrays: rows outside x and y are not touched."""
    T, K, N, n, r = 40, 64, 96, 3, 8
    s = _make(T, K, N, n, r, "f16", seed=2, ranks="full")
    p = S.RoutePlan(T, 1, n)
    rng = np.random.default_rng(4)
    for arr in (p.order, p.offsets, p.tiles):
        bad = rng.choice([-2 ** 31, -7, 0, 5, 39, 40, 1000, 2 ** 31 - 1], arr.numel()).astype(np.int32)
        arr.copy_(torch.from_numpy(bad).cuda().view(arr.shape))
    yb = torch.full((T + 2, N), -3.0, device="cuda")
    for fn in (lambda: S.lora_apply(s["ranks_t"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"], None,
                                    yb[1:T + 1], s["ws"]),
               lambda: S.lora_grad(s["ranks_t"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"],
                                   torch.zeros(T, N, device="cuda").half(), torch.empty(n, r, K, device="cuda"),
                                   torch.empty(n, r, N, device="cuda"), s["ws"])):
        fn()
        torch.cuda.synchronize()
        assert (yb[0] == -3).all() and (yb[T + 1] == -3).all()


def test_refusals_of_shapes():
    s = _make(8, 64, 64, 2, 8, "f16", seed=1)
    y = torch.zeros(8, 64, device="cuda")
    p = s["plan"]
    other = S.RoutePlan(9, 1, 2)
    call = lambda **k: S.lora_apply(k.get("ranks", s["ranks_t"]), s["scale"], k.get("A", s["A"]), k.get("B", s["B"]),  # noqa: E731
                                    k.get("order", p.order), p.offsets, p.tiles, k.get("x", s["x"]), None, k.get("y", y), s["ws"])
    for kw, err in ((dict(order=other.order), ValueError), (dict(A=s["A"][:1]), ValueError), (dict(A=s["A"].float()), TypeError),
                    (dict(B=s["B"].transpose(1, 2)), ValueError), (dict(x=s["x"][:7]), ValueError),
                    (dict(y=y[:, :63]), ValueError), (dict(y=y.bfloat16()), TypeError),
                    (dict(ranks=s["ranks_t"][:1]), ValueError), (dict(x=s["x"].float()), TypeError)):
        with pytest.raises(err):
            call(**kw)
