"""The order in which the embedding gradient adds: tokens of an id that lie in one block
of 16 sorted positions are summed one after another, in the tokens' order, by either sort."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")


def _batch(n, vocab, width, seed):
    """ids of 3 to 7 tokens each mostly, dy over 16 powers of two; rows {id: tokens} in one block of 16."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, vocab, n).astype(np.int32)
    dy = (rng.standard_normal((n, width)) * 2.0 ** rng.integers(-8, 9, (n, 1))).astype(np.float32)
    order = np.argsort(ids, kind="stable")
    starts = np.searchsorted(ids[order], np.arange(vocab + 1))
    rows = {v: order[a:b] for v, (a, b) in enumerate(zip(starts[:-1], starts[1:])) if b - a >= 3 and a // 16 == (b - 1) // 16}
    return ids, dy, rows


def _sum(dy):
    s = np.zeros(dy.shape[1], np.float32)
    for row in dy:
        s = s + row
    return s


@pytest.mark.parametrize("n", [900, 16384, 16385, 40000])
def test_the_sums_depend_on_the_order(n):
    _, dy, rows = _batch(n, n // 5, 24, n)
    assert len(rows) > n // 20
    other = sum(not np.array_equal(_sum(dy[at]), _sum(dy[at[::-1]])) for at in rows.values())
    assert other > 0.9 * len(rows)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [900, 16384, 16385, 40000])
def test_tokens_are_added_in_their_order(n):
    ids, dy, rows = _batch(n, n // 5, 24, n)
    out = torch.empty(n // 5, 24, device="cuda")
    ws = torch.empty(S.embed_grad_workspace_size(n, n // 5, 24), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    S.embed_grad(torch.from_numpy(ids).cuda(), torch.from_numpy(dy).cuda(), out, ws)
    got = out.cpu().numpy()
    for v, at in rows.items():
        assert np.array_equal(got[v], _sum(dy[at])), v
