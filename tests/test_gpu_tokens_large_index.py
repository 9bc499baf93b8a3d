"""Rows whose element offsets pass 2^31 (and byte offsets 2^32): the many-token
operators on wide-strided views of large buffers, compared with the same call
on packed copies, bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

from helpers import dev  # noqa: E402

pytestmark = pytest.mark.gpu

LD, T = 1 << 20, 2100                      # 2100 rows 2^20 elements apart: 2.2e9 elements


def _far(width, dtype, like=None):
    """[T, width] view with row stride LD, zeros or a copy of `like`."""
    v = torch.empty(T * LD, dtype=dtype, device="cuda").view(T, LD)[:, :width]
    if like is None:
        v.fill_(0)
    else:
        v.copy_(like)
    assert v.stride(0) * (T - 1) > 2 ** 31
    return v


def test_routing():
    d, e = 264, 7
    keys = torch.from_numpy(np.random.default_rng(0).integers(-1, e, (T, 1)).astype(np.int32)).cuda()
    p = S.RoutePlan(T, 1, e).build(keys)
    x, w = torch.randn(T, d, device="cuda").bfloat16(), torch.rand(T, 1, device="cuda")
    xs = p.gather(x, torch.zeros_like(x))
    far = p.gather(_far(d, x.dtype, x), _far(d, x.dtype))
    assert torch.equal(far, xs)
    assert torch.equal(p.combine(far, _far(d, x.dtype), w), p.combine(xs, torch.empty_like(x), w))
    a, b = p.combine_grad(_far(d, x.dtype, x), far, w, _far(d, x.dtype), torch.empty_like(w))
    c, f = p.combine_grad(x, xs, w, torch.zeros_like(x), torch.empty_like(w))
    assert torch.equal(a, c) and torch.equal(b, f)


def test_adapters():
    K, N, n, r = 136, 520, 3, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    half = lambda *sh: torch.randn(*sh, device="cuda", generator=g).half()  # noqa: E731
    A, B, x, base, dy = half(n, r, K), half(n, r, N), half(T, K), half(T, N), half(T, N)
    keys = torch.from_numpy(np.random.default_rng(0).integers(-1, n, T).astype(np.int32)).cuda()
    p = S.RoutePlan(T, 1, n).build(keys)
    ws = torch.empty(S.lora_workspace_size(T, r), dtype=torch.uint8, device="cuda")
    call = lambda x, b, y: S.lora_apply(None, None, A, B, p.order, p.offsets, p.tiles, x, b, y, ws)  # noqa: E731
    want = call(x, base, torch.empty_like(base))
    assert torch.equal(call(_far(K, x.dtype, x), _far(N, x.dtype, base), _far(N, x.dtype)), want)
    grad = lambda x, dy: S.lora_grad(None, None, A, B, p.order, p.offsets, p.tiles, x, dy,  # noqa: E731
                                     torch.empty(n, r, K, device="cuda"), torch.empty(n, r, N, device="cuda"), ws)
    for a, b in zip(grad(_far(K, x.dtype, x), _far(N, x.dtype, dy)), grad(x, dy)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [520, 521])
def test_pruned_product(cols):
    rows = 96
    rng = np.random.default_rng(2)
    dense = np.where(rng.random((rows, cols)) < 0.4, rng.standard_normal((rows, cols)), 0).astype(np.float16)
    rp = np.concatenate([[0], np.cumsum((dense != 0).sum(1))]).astype(np.int32)
    mrp, codes, mv = S.macko_encode(rows, cols, rp, np.nonzero(dense)[1].astype(np.int32), dense[dense != 0].view(np.uint16))
    m = S.MackoMatrix(rows, cols, dev(mrp), dev(codes.view(np.int32)), dev(mv.view(np.float16)))
    x = torch.randn(T, cols, device="cuda").half()
    want = m.apply(x, torch.empty(T, rows, device="cuda"))
    assert torch.equal(m.apply(_far(cols, x.dtype, x), _far(rows, torch.float32)), want)
