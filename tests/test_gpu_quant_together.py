"""A small model's step on 4-bit weights as a program runs it: token rows looked
up, a projection, a layer of experts on top, the logits; beside it the table's
gradient.  Each step against 64 bits from its own inputs, and the whole, captured
in one graph, replayed to the same bits as the eager calls."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
import quant_refs as Q  # noqa: E402

pytestmark = pytest.mark.gpu

VOCAB, D, INTER, E, GROUP = 1003, 264, 200, 6, 64


class Model:
    def __init__(self, T, k, dt, zeros, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.k, self.dt = T, k, dt
        w = lambda rows, cols, i: Q.weight(rows, cols, GROUP, dt, zeros, seed + i, scale=0.4 / cols ** 0.5)  # noqa: E731
        raw = [w(D, D, 1), w(E * 2 * INTER, D, 2), w(E * D, INTER, 3), w(VOCAB, D, 4)]
        dev = [[None if t is None else t.cuda() for t in r] for r in raw]
        self.proj = S.Q4Matrix(D, D, *dev[0], group=GROUP)
        self.gu = S.Q4Matrix(2 * INTER, D, *dev[1], group=GROUP, n_groups=E)
        self.dn = S.Q4Matrix(D, INTER, *dev[2], group=GROUP, n_groups=E)
        self.head = S.Q4Matrix(VOCAB, D, *dev[3], group=GROUP)
        self.proj64, self.head64 = Q.dense(*raw[0], GROUP, D), Q.dense(*raw[3], GROUP, D)
        self.up64 = Q.dense(*raw[1], GROUP, D).view(E, 2 * INTER, D)
        self.dn64 = Q.dense(*raw[2], GROUP, INTER).view(E, D, INTER)
        new = lambda *sh, t=dt: torch.zeros(*sh, dtype=t, device="cuda")  # noqa: E731
        self.table = (torch.randn(VOCAB, D, device="cuda", generator=g) * 0.02).to(dt)
        self.dy = torch.randn(T, D, device="cuda", generator=g).to(dt)
        self.ids, self.keys = new(T, t=torch.int32), new(T, k, t=torch.int32)
        self.w = torch.rand(T, k, device="cuda", generator=g)
        self.x, self.h, self.y = new(T, D), new(T, D), new(T, D)
        self.logits, self.dtable = new(T, VOCAB, t=torch.float32), new(VOCAB, D, t=torch.float32)
        ws = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws_p, self.ws_h = self.proj.workspace(T), self.head.workspace(T)
        self.ws_m = ws(S.moe_workspace_size(T, k, D, INTER))
        self.ws_e = ws(S.embed_grad_workspace_size(T, VOCAB, D))
        self.set_batch(seed)

    def set_batch(self, seed):
        rng = np.random.default_rng(seed)
        self.ids.copy_(torch.from_numpy(rng.zipf(1.3, self.T).astype(np.int64) % (VOCAB + 3) - 1))
        self.keys.copy_(torch.from_numpy(rng.integers(-1, E, (self.T, self.k))))

    def step(self):
        S.embed_lookup(self.ids, self.table, self.x, scale=16.0)
        self.proj.apply(self.x, self.h, workspace=self.ws_p)
        S.moe_apply(self.keys, self.w, self.gu, self.dn, self.h, self.y, self.ws_m)
        self.head.apply(self.y, self.logits, workspace=self.ws_h)
        S.embed_grad(self.ids, self.dy, self.dtable, self.ws_e, scale=16.0)

    def results(self):
        return [t.clone() for t in (self.x, self.h, self.y, self.logits, self.dtable)]


@pytest.mark.parametrize("T,k,dt,zeros", [(1, 2, torch.float16, False), (7, 2, torch.bfloat16, True),
                                          (40, 3, torch.float16, True), (150, 2, torch.bfloat16, False)])
def test_step(T, k, dt, zeros):
    m = Model(T, k, dt, zeros, seed=T)
    m.step()
    torch.cuda.synchronize()
    ref, bound = Q.embed(m.ids.cpu().numpy(), m.table, 16.0, dt)
    R.check(m.x, ref, bound, "rows")
    ref, bound = Q.matmul(m.proj64, m.x, 1.0, 0.0, None, dt, GROUP)
    R.check(m.h, ref, bound, "projection")
    ref, bound = Q.moe(m.keys.cpu(), m.w.cpu(), m.up64, m.dn64, m.h, dt, GROUP)
    R.check(m.y, ref, bound, "experts")
    ref, bound = Q.matmul(m.head64, m.y, 1.0, 0.0, None, torch.float32, GROUP)
    R.check(m.logits, ref, bound, "logits")
    ref, bound = Q.embed_grad(m.ids.cpu().numpy(), m.dy, VOCAB, 16.0)
    R.check(m.dtable, ref, bound, "gradient")


@pytest.mark.parametrize("T", [6, 70])
def test_step_replayed_from_a_graph(T):
    m, other = Model(T, 2, torch.bfloat16, True, seed=3), Model(33, 2, torch.float16, False, seed=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    scratch = (m.x, m.h, m.y, m.logits, m.dtable)
    for i in range(4):
        m.set_batch(20 + i)
        m.dy.copy_(torch.randn(T, D, device="cuda"))
        for t in scratch:
            t.fill_(float("nan"))
        for t in (m.ws_p, m.ws_h, m.ws_m, m.ws_e):
            t.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        other.step()
        torch.cuda.synchronize()
        got = m.results()
        for t in scratch:
            t.fill_(float("nan"))
        m.step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, m.results())), i


def test_steps_on_two_streams_at_once():
    """Weights and tables are shared, outputs and workspaces are not."""
    a, b = Model(24, 2, torch.float16, True, seed=5), Model(24, 2, torch.float16, True, seed=5)
    for name in ("proj", "gu", "dn", "head", "table"):
        setattr(b, name, getattr(a, name))
    b.set_batch(99)
    a.step()
    b.step()
    torch.cuda.synchronize()
    want = a.results() + b.results()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for t in (a.logits, b.logits, a.dtable, b.dtable):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        for m, s in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(s):
                m.step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, a.results() + b.results()))
