"""4-bit products, expert layers and embeddings past 32-bit offsets: strides of
2^31 elements, arranged weights of more than 4 GB, tables of more than 2^32 bytes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
import quant_refs as Q  # noqa: E402

pytestmark = pytest.mark.gpu


def _far(n, width, dt):
    """n rows 2^31 + 8 elements apart (memory that is never touched between them)."""
    return torch.empty((n - 1) * (2 ** 31 + 8) + width, dtype=dt, device="cuda").as_strided((n, width), (2 ** 31 + 8, 1))


@pytest.mark.parametrize("tok", [2, 4, 6])
def test_q4_rows_far_apart(tok):
    rows, cols, dt = 40, 200, torch.float16
    w = Q.weight(rows, cols, 64, dt, True, 1)
    m = S.Q4Matrix(rows, cols, *[t.cuda() for t in w], group=64)
    x, y = _far(tok, cols, dt), _far(tok, rows, dt)
    x.copy_(torch.randn(tok, cols))
    m.apply(x, y)
    ref, bound = Q.matmul(Q.dense(*w, 64, cols), x, 1.0, 0.0, None, dt, 64)
    R.check(y, ref, bound)


@pytest.mark.parametrize("tok", [1, 5, 40])
def test_q4_tiles_past_4_gb(tok):
    """A weight of 65552 x 131072: 4.5 GB of records.  Codes are the zero point but in the last rows."""
    rows, cols = 65552, 131072
    codes = torch.full((rows, cols // 8), -2004318072, dtype=torch.int32, device="cuda")          # 0x88888888
    g = torch.Generator().manual_seed(tok)
    last = torch.randint(0, 16, (16, cols), generator=g)
    codes[-16:] = Q.pack(last.numpy()).cuda()
    scales = torch.full((rows, cols // 128), 0.0625, dtype=torch.bfloat16, device="cuda")
    m = S.Q4Matrix(rows, cols, codes, scales)
    del codes
    assert m.tiles.numel() > 2 ** 32
    x = torch.randn(tok, cols, generator=g).bfloat16()
    y = m.apply(x.cuda(), torch.empty(tok, rows, device="cuda"))
    assert (y[:, :-16] == 0).all()
    ref, bound = Q.matmul((last.double() - 8) * 0.0625, x, 1.0, 0.0, None, torch.float32, 128)
    R.check(y[:, -16:], ref, bound)


def test_moe_rows_far_apart():
    dim, inter, e, dt = 72, 40, 3, torch.bfloat16
    up, dn = Q.weight(e * 2 * inter, dim, 32, dt, False, 1), Q.weight(e * dim, inter, 32, dt, False, 2)
    gu = S.Q4Matrix(2 * inter, dim, up[0].cuda(), up[1].cuda(), None, group=32, n_groups=e)
    dm = S.Q4Matrix(dim, inter, dn[0].cuda(), dn[1].cuda(), None, group=32, n_groups=e)
    x, y = _far(3, dim, dt), _far(3, dim, dt)
    x.copy_(torch.randn(3, dim))
    for k in (2, 30):                                        # either form of the down product
        keys = torch.randint(-1, e, (3, k), dtype=torch.int32)
        w = torch.rand(3, k)
        S.moe_apply(keys.cuda(), w.cuda(), gu, dm, x, y,
                    torch.empty(S.moe_workspace_size(3, k, dim, inter), dtype=torch.uint8, device="cuda"))
        ref, bound = Q.moe(keys, w, Q.dense(*up, 32, dim).view(e, 2 * inter, dim), Q.dense(*dn, 32, inter).view(e, dim, inter),
                           x, dt, 32)
        R.check(y, ref, bound, f"{k} choices")


def test_embed_past_4_gb():
    v, d = 2 ** 20 + 77, 2100                                # 4.4 GB in fp16, 8.8 GB of gradient
    table = torch.zeros(v, d, dtype=torch.float16, device="cuda")
    ids = np.array([v - 1, 5, v - 2, v - 1, 2 ** 20, -1, v], np.int32)
    at = torch.from_numpy(np.unique(ids[(ids >= 0) & (ids < v)]).astype(np.int64)).cuda()
    table[at] = torch.randn(len(at), d, device="cuda").half()
    y = S.embed_lookup(torch.from_numpy(ids).cuda(), table, torch.empty(7, d, device="cuda"), scale=0.5)
    for i, t in enumerate(ids):
        want = 0.5 * table[int(t)].float() if 0 <= t < v else torch.zeros(d, device="cuda")
        assert torch.equal(y[i], want), i
    del table
    dy = torch.randn(7, d, device="cuda")
    out = torch.full((v, d), float("nan"), device="cuda")
    ws = torch.empty(S.embed_grad_workspace_size(7, v, d), dtype=torch.uint8, device="cuda")
    S.embed_grad(torch.from_numpy(ids).cuda(), dy, out, ws)
    assert torch.equal(out[v - 1], dy[0] + dy[3]) and torch.equal(out[v - 2], dy[2])
    assert torch.equal(out[2 ** 20], dy[4]) and torch.equal(out[5], dy[1])
    out[at] = 0.0
    assert out.abs().max().item() == 0.0
    S.embed_grad(torch.from_numpy(ids).cuda(), dy, out, ws, accumulate=True)
    assert torch.equal(out[v - 1], dy[0] + dy[3])
