"""How many bits of the rank vectors the adapters' kernels keep: tokens, ranks
and tiles of very different size beside each other, against 64 bits.  Each
entry of a rank vector counts with its own size in the bounds, never with
that of a larger neighbour."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402

pytestmark = pytest.mark.gpu

F = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


def _plan(keys, n):
    return S.RoutePlan(len(keys), 1, n).build(torch.from_numpy(np.asarray(keys, np.int32)).cuda())


def _randn(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *sh: torch.randn(*sh, device="cuda", generator=g)


# ---------------------------------------------------------------------------
# Weight gradients
# ---------------------------------------------------------------------------
def _grad(A, B, x, dy, keys=None):
    n, r, _ = A.shape
    p = _plan(np.zeros(x.shape[0]) if keys is None else keys, n)
    dA, dB = (torch.full(t.shape, NAN, device="cuda") for t in (A, B))
    ws = torch.full((S.lora_workspace_size(x.shape[0], r),), 255, dtype=torch.uint8, device="cuda")
    S.lora_grad(None, None, A, B, p.order, p.offsets, p.tiles, x, dy, dA, dB, ws)
    torch.cuda.synchronize()
    return dA, dB


def _check_grad(A, B, x, dy, keys=None, what=""):
    """dA[a, j, k] = sum_t g_tj x_tk with g = dy B^T, and dB the same with x and
    dy, A and B exchanged.  g: chains of at most K / 32 + 32 additions and 40
    partial sums; as an operand 2^-23 of each entry's own size.  The sum over
    tokens: at most 6 instructions per 32 tokens, each adding up 32 products
    (counted as 32 additions once and one per instruction), 16 partial sums."""
    dA, dB = _grad(A, B, x, dy, keys)
    keys = np.zeros(x.shape[0]) if keys is None else np.asarray(keys)
    for got, W, u, v, name in ((dA, B, dy, x, "dA"), (dB, A, x, dy, "dB")):
        W, u, v = R.f64(W), R.f64(u), R.f64(v)
        for a in range(W.shape[0]):
            at = torch.from_numpy(np.flatnonzero(keys == a))
            g = u[at] @ W[a].t()
            dg = (u[at].abs() @ W[a].abs().t()) * ((u.shape[1] / 32 + 72) * R.ADD) + g.abs() * 2.0 ** -23
            mag = (g.abs() + dg).t() @ v[at].abs()
            bound = dg.t() @ v[at].abs() + mag * ((32 + 6 * (len(at) / 32 + 1) + 16) * R.ADD)
            R.check(got[a], g.t() @ v[at], bound, f"{what} {name} of adapter {a}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N,r", [(20, 128, 72, 8), (700, 264, 136, 8), (300, 1040, 520, 16), (8200, 64, 72, 16)])
def test_grad_with_ranks_of_different_size(T, K, N, r, dt):
    """The rows of A and B each 8 times smaller than the one before."""
    randn = _randn(T)
    fall = torch.tensor([8.0 ** -(j % 8) for j in range(r)], device="cuda")[None, :, None]
    _check_grad(((randn(1, r, K) * fall)).to(F[dt]), (randn(1, r, N) * fall).to(F[dt]), randn(T, K).to(F[dt]),
                randn(T, N).to(F[dt]))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("big", [0, 17, 299])
def test_grad_with_one_large_token(big, dt):
    """One token's rows 2^18 above the others', with columns that only the others use."""
    T, K, N, r = 300, 136, 264, 8
    randn = _randn(big)
    size = torch.full((T, 1), 2.0 ** -12, device="cuda")
    size[big] = 2.0 ** 6
    x, dy = randn(T, K), randn(T, N)
    for large, other in ((dy, x), (x, dy)):
        a, b = large * size, other.clone()
        b[big, ::2] = 0
        xx, dd = (b, a) if large is dy else (a, b)
        _check_grad(randn(1, r, K).to(F[dt]), randn(1, r, N).to(F[dt]), xx.to(F[dt]), dd.to(F[dt]))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("K,N,r", [(64, 72, 8), (520, 264, 40), (7, 135, 20)])
def test_grad_of_tiles_far_apart(K, N, r, dt):
    """Tiles of 16 tokens 2^26 apart, in both orders, and columns that only the small ones use."""
    randn = _randn(K)
    for order in (0, 1):
        x, dy = randn(64, K), randn(64, N)
        for t in range(0, 64, 16):
            small = (t // 16 + order) % 2 == 0
            dy[t:t + 16] *= 2.0 ** -14 if small else 2.0 ** 12
            if not small:
                x[t:t + 16, ::2] = 0
        A, B = randn(2, r, K).to(F[dt]), randn(2, r, N).to(F[dt])
        keys = np.r_[np.zeros(40), np.ones(24)]
        _check_grad(A, B, x.to(F[dt]), dy.to(F[dt]), keys)
        _check_grad(B, A, dy.to(F[dt]), x.to(F[dt]), keys)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_grad_of_exact_rank_vectors(dt):
    """Columns with one entry in A and B: rank vectors are single products, so
    only the operand's rounding and the sum over tokens are left.  Token t's
    rank vector is 2^(t mod 20) times another's; x gives them all one size."""
    T, r = 160, 8
    randn = _randn(3)
    up = torch.tensor([2.0 ** (t % 20 - 10) for t in range(T)], device="cuda")[:, None]
    A = torch.zeros(1, r, r, device="cuda")
    B = torch.zeros(1, r, r, device="cuda")
    for j in range(r):
        A[0, j, j], B[0, j, j] = 1 + j / 8, 2.0 ** -j * (1 + j / 16)
    A, B, x, dy = (t.to(F[dt]) for t in (A, B, randn(T, r) / up, randn(T, r) * up))
    dA, dB = _grad(A, B, x, dy)
    for got, W, u, v in ((dA, B, dy, x), (dB, A, x, dy)):
        g, v = R.f64(u) @ R.f64(W)[0].t(), R.f64(v)
        R.check(got[0], g.t() @ v, (g.abs().t() @ v.abs()) * (2.0 ** -23 + (32 + 6 * (T / 32 + 1) + 16) * R.ADD))


# ---------------------------------------------------------------------------
# The adapters' product
# ---------------------------------------------------------------------------
def _check_apply(A, B, x, y_in, ydt, what=""):
    """y = y_in + B^T (A x).  h = A x: chains of at most K / 32 + 32 additions and
    40 partial sums; as an operand all 24 bits (2^-25 of each entry's own size); then
    at most three terms of r products, and 24 more sums and products."""
    n, r, K = A.shape
    T, N = x.shape[0], B.shape[2]
    keys = (np.arange(T) + 1) % (n + 1) - 1
    p = _plan(keys, n)
    ws = torch.full((S.lora_workspace_size(T, r),), 255, dtype=torch.uint8, device="cuda")
    y = torch.full((T, N), NAN, device="cuda", dtype=ydt)
    base = None if y_in is None else y_in.to(ydt)
    S.lora_apply(None, None, A, B, p.order, p.offsets, p.tiles, x, base, y, ws)
    torch.cuda.synchronize()
    ref = torch.zeros(T, N, dtype=torch.float64) if base is None else R.f64(base).clone()
    bound = torch.zeros(T, N, dtype=torch.float64)
    A, B, x = R.f64(A), R.f64(B), R.f64(x)
    for a in range(n):
        at = torch.from_numpy(np.flatnonzero(keys == a))
        h = x[at] @ A[a].t()
        dh = (x[at].abs() @ A[a].abs().t()) * ((K / 32 + 72) * R.ADD) + h.abs() * 2.0 ** -25
        mag = (h.abs() + dh) @ B[a].abs()
        ref[at] += h @ B[a]
        bound[at] = dh @ B[a].abs() + mag * ((3 * r + 24) * R.ADD) + ref[at].abs() * 2 * R.ADD
    R.check(y, ref, bound + R.rounded(ref.abs() + bound, ydt), what)


def _spread(T, K, N, r, lo, hi, seed):
    """Adapters whose rank vectors hold entries of very different size, in another
    order for every token, beside columns of B that take one rank each: rank j
    reads the columns of x with k mod r = j, whose size is 2^s."""
    rng = np.random.default_rng(seed)
    randn = _randn(seed)
    s = torch.from_numpy(rng.uniform(lo, hi, (T, r))).cuda()
    col = torch.arange(K, device="cuda") % r
    x = randn(T, K) * torch.exp2(torch.round(s))[:, col]
    A = randn(2, r, K) * (col[None, None, :] == torch.arange(r, device="cuda")[None, :, None])
    B = randn(2, r, N) * (torch.arange(N, device="cuda")[None, None, :] % r == torch.arange(r, device="cuda")[None, :, None])
    return A, B, x


@pytest.mark.parametrize("y", ["x", "f32"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N,r", [(1, 128, 72, 8), (37, 264, 1032, 8), (20, 520, 130, 24), (300, 136, 264, 40), (33, 200, 515, 100)])
def test_apply_with_ranks_of_different_size(T, K, N, r, dt, y):
    """The rows of A each 8 times smaller than the one before, those of B larger."""
    randn = _randn(T)
    step = torch.tensor([8.0 ** (j % 8) for j in range(r)], device="cuda")[None, :, None]
    ydt = F[dt] if y == "x" else torch.float32
    A, B = (randn(2, r, K) / step).to(F[dt]), (randn(2, r, N) * step / 1024).to(F[dt])
    _check_apply(A, B, randn(T, K).to(F[dt]), randn(T, N), ydt)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N,r", [(1, 64, 64, 4), (18, 8, 8, 8), (50, 264, 515, 16), (35, 260, 1032, 20), (300, 200, 264, 33), (40, 512, 200, 128),
                                     (20, 7, 5, 3)])
def test_apply_with_entries_far_apart(T, K, N, r, dt):
    """Rank vectors with entries up to 2^60 apart."""
    A, B, x = _spread(T, K, N, r, -13, 14, seed=T + r)
    up = torch.exp2(torch.round(torch.linspace(-12, 14, r, device="cuda")))[None, :, None]
    _check_apply((A * up).to(F[dt]), B.to(F[dt]), x.to(F[dt]), None, torch.float32, "far")
    _check_apply((A * up).to(F[dt]), B.to(F[dt]), x.to(F[dt]), _randn(2)(T, N), torch.float32, "far, added")
    A, B, x = _spread(T, K, N, r, -3, 14, seed=T + r)
    _check_apply((A / 256).to(F[dt]), B.to(F[dt]), x.to(F[dt]), _randn(2)(T, N), F[dt], "rounded")


@pytest.mark.parametrize("y", ["x", "f32"])
@pytest.mark.parametrize("r", [2, 40])
def test_apply_where_ranks_cancel(r, y):
    """bf16 rank vectors of 24 bits, exact in fp32 (two products each), whose
    neighbours differ by 2^-15 and meet rows of B of opposite sign: what is left
    shows every bit of the operand."""
    T, N = 64, 136
    rng = np.random.default_rng(r)
    A = torch.zeros(1, r, 2, device="cuda")
    one = 1 + torch.from_numpy(rng.integers(0, 128, (r // 2, 2)) / 128).float()
    A[0, 0::2] = A[0, 1::2] = one.cuda()
    A[0, 1::2, 1] += torch.where(A[0, 1::2, 1] < 1.9, 2.0 ** -7, -2.0 ** -7)
    B = _randn(5)(1, r, N)
    B[0, 1::2] = -B[0, 0::2]
    x = 1 + torch.from_numpy(rng.integers(0, 128, (T, 2)) / 128).float().cuda()
    x[:, 1] *= 2.0 ** -8
    A, B, x = A.bfloat16(), B.bfloat16(), x.bfloat16()
    h = R.f64(x) @ R.f64(A)[0].t()
    assert torch.equal(h, h.float().double())
    p = _plan(np.zeros(T), 1)
    out = torch.full((T, N), NAN, device="cuda", dtype=F["bf16"] if y == "x" else torch.float32)
    S.lora_apply(None, None, A, B, p.order, p.offsets, p.tiles, x, None, out,
                 torch.empty(S.lora_workspace_size(T, r), dtype=torch.uint8, device="cuda"))
    ref = h @ R.f64(B)[0]
    bound = (h.abs() @ R.f64(B)[0].abs()) * ((3 * r + 6) * R.ADD)
    R.check(out, ref, bound + R.rounded(ref.abs() + bound, out.dtype), "cancelled")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("r", [1, 20, 100])
def test_rows_of_one_give_the_rank_vector_itself(r, dt):
    """B holds the unit rows, so y is A x: sums of two products that fill fp32's
    24 bits come back exactly."""
    T = 50
    rng = np.random.default_rng(r)
    step = 1024 if dt == "f16" else 128                  # a type's last bit of 1.xx
    mant = lambda *sh: torch.from_numpy(1 + rng.integers(0, step * 2 // 5, sh) / step).cuda()  # noqa: E731
    A, x = mant(1, r, 2), mant(T, 2)
    x[:, 1] *= 2.0 ** (-2 if dt == "f16" else -8)
    x *= torch.exp2(torch.arange(T, device="cuda") % 21 - 10.0)[:, None]
    A, x, B = A.to(F[dt]), x.to(F[dt]), torch.eye(r, device="cuda")[None].to(F[dt])
    h = R.f64(x) @ R.f64(A)[0].t()
    assert torch.equal(h, h.float().double())
    p = _plan(np.zeros(T), 1)
    y = torch.full((T, r), NAN, device="cuda")
    S.lora_apply(None, None, A, B, p.order, p.offsets, p.tiles, x, None, y,
                 torch.empty(S.lora_workspace_size(T, r), dtype=torch.uint8, device="cuda"))
    assert torch.equal(R.f64(y), h)


# ---------------------------------------------------------------------------
# Infinities
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("N,r", [(64, 1), (265, 8), (72, 24), (136, 90), (7, 3)])
def test_apply_of_infinities(N, r, dt):
    """A token with an infinity gets infinities of the definition's signs, and NaN
    where it has NaN: where they meet zeros or each other."""
    T, K = 20, 72
    randn = _randn(N)
    A, B, x = randn(1, r, K).abs() + 0.25, randn(1, r, N), randn(T, K)
    B[0, :, ::3] = B[0, :, ::3].abs() + 0.25
    B[0, :, 1::9] = 0
    x[3, 5], x[7, 71], x[8, 0] = float("inf"), -float("inf"), NAN
    x[9, 1], x[9, 2] = float("inf"), -float("inf")
    A, B, x = A.to(F[dt]), B.to(F[dt]), x.to(F[dt])
    base = randn(T, N)
    p = _plan(np.zeros(T), 1)
    y = torch.empty(T, N, device="cuda")
    S.lora_apply(None, None, A, B, p.order, p.offsets, p.tiles, x, base, y,
                 torch.empty(S.lora_workspace_size(T, r), dtype=torch.uint8, device="cuda"))
    h = (R.f64(x)[:, None, :] * R.f64(A)[0]).sum(2)
    ref = R.f64(base) + (h[:, :, None] * R.f64(B)[0]).sum(1)
    got = R.f64(y)
    for t in (3, 7, 8, 9):
        assert torch.equal(torch.isnan(got[t]), torch.isnan(ref[t])), t
        ok = ~torch.isnan(ref[t])
        assert torch.equal(got[t][ok], ref[t][ok]) and not torch.isfinite(ref[t]).any(), t
    rest = [t for t in range(T) if t not in (3, 7, 8, 9)]
    assert torch.isfinite(got[rest]).all()


def test_rank_vector_past_fp32_beside_a_finite_one():
    """bf16: one entry of A x overflows to an infinity, its neighbour is close to
    fp32's largest number and stays finite."""
    A = torch.zeros(1, 2, 8, device="cuda").bfloat16()
    A[0, 0, 0], A[0, 1, 1], A[0, 1, 2] = 2.0 ** 100, 2.0 ** 100, 2.0 ** 92
    x = torch.zeros(3, 8, device="cuda").bfloat16()
    x[0, 0] = 2.0 ** 100
    x[1, 1], x[1, 2] = 2.0 ** 28 - 2.0 ** 20, 2.0 ** 28 - 2.0 ** 20        # 2^128 - 2^112: rounds past bf16's largest
    x[2, 1] = 1.0
    B = torch.zeros(1, 2, 16, device="cuda").bfloat16()
    B[0, 0, :8], B[0, 1, 8:] = 2.0, 2.0 ** -20
    p = _plan(np.zeros(3), 1)
    y = torch.empty(3, 16, device="cuda")
    S.lora_apply(None, None, A, B, p.order, p.offsets, p.tiles, x, None, y,
                 torch.empty(S.lora_workspace_size(3, 2), dtype=torch.uint8, device="cuda"))
    h = (R.f64(x)[:, None, :] * R.f64(A)[0]).sum(2)
    assert h[1, 1] < 2.0 ** 128 and float(h[1, 1].float()) == float(h[1, 1])
    assert (y[0, :8] == float("inf")).all() and torch.isnan(y[0, 8:]).all()      # an infinity times zero
    assert (R.f64(y[1, 8:]) == h[1, 1] * 2.0 ** -20).all() and (y[1, :8] == 0).all()
    assert (y[2, 8:] == 2.0 ** 80).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_grad_of_infinities(dt):
    """What a bad element takes part in is not finite, the rest is as without it."""
    T, K, N, n, r = 100, 72, 136, 3, 20
    randn = _randn(9)
    A, B, x, dy = (t.to(F[dt]) for t in (randn(n, r, K), randn(n, r, N), randn(T, K), randn(T, N)))
    keys = np.arange(T) % n
    dA0, dB0 = _grad(A, B, x, dy, keys)
    for bad in (float("inf"), NAN):
        xb, db = x.clone(), dy.clone()
        xb[7, 5] = bad                     # adapter 1
        db[11, 130] = bad                  # adapter 2
        dA, dB = _grad(A, B, xb, db, keys)
        assert torch.equal(dA[0], dA0[0]) and torch.equal(dB[0], dB0[0])
        keep = [k for k in range(K) if k != 5]
        assert torch.equal(dA[1][:, keep], dA0[1][:, keep]) and not torch.isfinite(dA[1][:, 5]).any()
        assert not torch.isfinite(dB[1]).any()
        keep = [k for k in range(N) if k != 130]
        assert torch.equal(dB[2][:, keep], dB0[2][:, keep]) and not torch.isfinite(dB[2][:, 130]).any()
        assert not torch.isfinite(dA[2]).any()


def test_grad_without_tokens_or_workspace():
    A, B = torch.ones(3, 8, 64, device="cuda").half(), torch.ones(3, 8, 72, device="cuda").half()
    p = _plan([], 3)
    dA, dB = torch.full(A.shape, NAN, device="cuda"), torch.full(B.shape, NAN, device="cuda")
    x, dy = A[0, :0], B[0, :0]
    S.lora_grad(None, None, A, B, p.order, p.offsets, p.tiles, x, dy, dA, dB, None)
    assert (dA == 0).all() and (dB == 0).all()
    assert S.lora_apply(None, None, A, B, p.order, p.offsets, p.tiles, x, None, dy, None) is dy


@pytest.mark.parametrize("low", [-60, -104, -118, -124])
def test_rank_vectors_near_the_smallest_numbers(low):
    """bf16: entries of A x of 2^low come back through unit rows of B, and through the
    gradients, to 24 bits or to multiples of bf16's smallest number, 2^-133."""
    T, r = 40, 8
    rng = np.random.default_rng(-low)
    mant = lambda *sh: torch.from_numpy(1 + rng.integers(0, 51, sh) / 128).cuda()  # noqa: E731
    A, x = mant(1, r, 2) * 2.0 ** (low // 2), mant(T, 2) * 2.0 ** (low - low // 2)
    x[:, 1] *= 2.0 ** -8
    A, x, B = A.bfloat16(), x.bfloat16(), torch.eye(r, device="cuda")[None].bfloat16()
    h = R.f64(x) @ R.f64(A)[0].t()
    p = _plan(np.zeros(T), 1)
    y = torch.full((T, r), NAN, device="cuda")
    S.lora_apply(None, None, A, B, p.order, p.offsets, p.tiles, x, None, y,
                 torch.empty(S.lora_workspace_size(T, r), dtype=torch.uint8, device="cuda"))
    # the products' own last bits in fp32, and the operand's
    R.check(y, h, h.abs() * 2.0 ** -24 + 2.0 ** -149 + 2.0 ** -134, "apply")
    dy = torch.zeros(T, r, device="cuda").bfloat16()
    dy[3, 2] = 1.0
    dA, dB = _grad(A, B, x, dy)
    R.check(dB[0, :, 2], h[3], h[3].abs() * 2.0 ** -24 + 2.0 ** -149 + 2.0 ** -134, "dB")
