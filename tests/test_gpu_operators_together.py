"""The many-token operators as a program runs them: a layer of pruned experts
(router plan, tokens sorted, one MACKO weight per expert, results brought back
with their weights) beside a shared pruned projection with low-rank adapters,
forward and backward.  Every step is checked against 64 bits from the step's
own inputs, and the whole layer, captured in one graph, replays to the same
bits as the eager calls."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
from helpers import dev  # noqa: E402

pytestmark = pytest.mark.gpu

D, H, E, ADAPTERS, RANK = 264, 392, 5, 3, 16


def _weight(rng, rows, cols, groups, keep):
    """(MackoMatrix, its transpose's, dense float64 [groups, rows, cols]), values exact in fp16."""
    dense = np.where(rng.random((groups, rows, cols)) < keep, rng.integers(1, 64, (groups, rows, cols)) / 1024.0, 0.0)
    dense *= rng.choice([-1, 1], dense.shape)

    def encode(w):
        flat = w.reshape(-1, w.shape[-1])
        rp = np.concatenate([[0], np.cumsum((flat != 0).sum(1))]).astype(np.int32)
        ci = np.nonzero(flat)[1].astype(np.int32)
        mrp, codes, mv = S.macko_encode(flat.shape[0], w.shape[-1], rp, ci, flat[flat != 0].astype(np.float16).view(np.uint16))
        return S.MackoMatrix(w.shape[1], w.shape[2], dev(mrp), dev(codes.view(np.int32)), dev(mv.view(np.float16)),
                             n_groups=groups)
    return encode(dense), encode(dense.transpose(0, 2, 1).copy()), torch.from_numpy(dense)


class Layer:
    """y = sum_c w[t, c] * Expert_c(x[t]) + P x[t] + adapters(x[t]), and its gradients."""

    def __init__(self, T, k, seed):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.k = T, k
        self.experts, self.experts_t, self.dense_e = _weight(rng, H, D, E, 0.4)
        self.shared, self.shared_t, self.dense_s = _weight(rng, H, D, 1, 0.3)
        half = lambda *sh: torch.randn(*sh, device="cuda", generator=g).half()  # noqa: E731
        self.A, self.B = half(ADAPTERS, RANK, D) / 16, half(ADAPTERS, RANK, H)
        self.ranks = torch.tensor([RANK, 5, 11], dtype=torch.int32, device="cuda")
        self.scale = torch.tensor([0.5, 2.0, 1.0], device="cuda")
        self.route, self.adapt = S.RoutePlan(T, k, E), S.RoutePlan(T, 1, ADAPTERS)
        self.keys = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        self.who = torch.zeros(T, dtype=torch.int32, device="cuda")
        self.x, self.w, self.dy = half(T, D), torch.rand(T, k, device="cuda", generator=g), half(T, H)
        self.lora_ws = torch.empty(S.lora_workspace_size(T, RANK), dtype=torch.uint8, device="cuda")
        z = lambda r, c, dt=torch.float16: torch.zeros(r, c, dtype=dt, device="cuda")  # noqa: E731
        self.xs, self.ys, self.dys, self.dxs = z(T * k, D), z(T * k, H), z(T * k, H), z(T * k, D)
        self.moe, self.y, self.dw = z(T, H), z(T, H), z(T, k, torch.float32)
        self.dx_moe, self.dx = z(T, D), z(T, D)
        self.dA = torch.zeros(ADAPTERS, RANK, D, device="cuda")
        self.dB = torch.zeros(ADAPTERS, RANK, H, device="cuda")
        self.ws = {id(m): m.workspace(n) for m, n in ((self.experts, T * k), (self.experts_t, T * k), (self.shared, T),
                                                     (self.shared_t, T))}
        self.set_batch(seed)

    def set_batch(self, seed):
        rng = np.random.default_rng(seed)
        self.keys.copy_(torch.from_numpy(rng.integers(-1, E - 1, (self.T, self.k)).astype(np.int32)))    # the last expert idle
        self.who.copy_(torch.from_numpy(rng.integers(-1, ADAPTERS, self.T).astype(np.int32)))

    def forward(self):
        p = self.route.build(self.keys)
        self.adapt.build(self.who)
        p.gather(self.x, self.xs)
        self.experts.apply(self.xs, self.ys, tok_offsets=p.offsets, workspace=self.ws[id(self.experts)])
        p.combine(self.ys, self.moe, self.w)
        self.y.copy_(self.moe)
        self.shared.apply(self.x, self.y, beta=1.0, workspace=self.ws[id(self.shared)])
        a = self.adapt
        S.lora_apply(self.ranks, self.scale, self.A, self.B, a.order, a.offsets, a.tiles, self.x, self.y, self.y, self.lora_ws)

    def backward(self):
        p, a = self.route, self.adapt
        p.combine_grad(self.dy, self.ys, self.w, self.dys, self.dw)
        self.experts_t.apply(self.dys, self.dxs, tok_offsets=p.offsets, workspace=self.ws[id(self.experts_t)])
        p.combine(self.dxs, self.dx_moe)
        self.dx.copy_(self.dx_moe)
        self.shared_t.apply(self.dy, self.dx, beta=1.0, workspace=self.ws[id(self.shared_t)])
        S.lora_apply(self.ranks, self.scale, self.B, self.A, a.order, a.offsets, a.tiles, self.dy, self.dx, self.dx, self.lora_ws)
        S.lora_grad(self.ranks, self.scale, self.A, self.B, a.order, a.offsets, a.tiles, self.x, self.dy, self.dA, self.dB,
                    self.lora_ws)

    def results(self):
        return [t.clone() for t in (self.y, self.dx, self.dw, self.dA, self.dB)]


@pytest.mark.parametrize("T,k", [(1, 2), (7, 2), (90, 3), (300, 1)])
def test_layer(T, k):
    m = Layer(T, k, seed=T)
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    offsets, order, pos, _ = R.route_plan(m.keys.cpu().numpy(), E)
    n = int(offsets[-1])
    tok = torch.from_numpy(order[:n]) // k
    x, w, dy = R.f64(m.x), R.f64(m.w).reshape(-1)[torch.from_numpy(order[:n])], R.f64(m.dy)
    ranks, scale = m.ranks.tolist(), m.scale.tolist()
    assert torch.equal(R.f64(m.xs)[:n], x[tok])

    def grouped(out, inp, dense, what):
        for g in range(E):
            a, b = int(offsets[g]), int(offsets[g + 1])
            ref, bound = R.spmm(dense[g], inp[a:b], 1.0, 0.0, None, torch.float16)
            R.check(out[a:b], ref, bound, f"{what} of expert {g}")
    grouped(m.ys, m.xs, m.dense_e, "output")
    ys = R.f64(m.ys)[:n] * w[:, None]
    moe, mag = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    moe.index_add_(0, tok, ys)
    mag.index_add_(0, tok, ys.abs())
    R.check(m.moe, moe, mag * (k * 2.0 ** -24) + R.rounded(moe.abs() + mag * 2.0 ** -20, torch.float16), "combined")
    # the shared projection on top of it (rounded to fp16), then the adapters in place
    ref, bound = R.spmm(m.dense_s[0], m.x, 1.0, 1.0, m.moe, torch.float16)
    full, more = R.lora(m.who.tolist(), ranks, scale, m.A, m.B, m.x, torch.zeros(T, H), 22, torch.float16)
    R.check(m.y, ref + full, bound + more + R.rounded(ref.abs() + full.abs() + bound + more, torch.float16), "layer")

    R.check(m.dys[:n], dy[tok] * w[:, None], (dy[tok] * w[:, None]).abs() * 2.0 ** -24 +
            R.rounded(dy[tok] * w[:, None], torch.float16), "dys")
    dw = torch.zeros(T * k, dtype=torch.float64)
    dmag = torch.zeros(T * k, dtype=torch.float64)
    at = torch.from_numpy(order[:n])
    dw[at] = (R.f64(m.ys)[:n] * dy[tok]).sum(1)
    dmag[at] = (R.f64(m.ys)[:n] * dy[tok]).abs().sum(1)
    R.check(m.dw.reshape(-1), dw, dmag * ((H + 2) * 2.0 ** -24), "dw")
    grouped(m.dxs, m.dys, m.dense_e.transpose(1, 2), "gradient")
    dx = torch.zeros(T, D, dtype=torch.float64)
    dxm = torch.zeros(T, D, dtype=torch.float64)
    dx.index_add_(0, tok, R.f64(m.dxs)[:n])
    dxm.index_add_(0, tok, R.f64(m.dxs)[:n].abs())
    R.check(m.dx_moe, dx, dxm * (k * 2.0 ** -24) + R.rounded(dx.abs() + dxm * 2.0 ** -20, torch.float16), "dx of the experts")
    ref, bound = R.spmm(m.dense_s[0].t().contiguous(), m.dy, 1.0, 1.0, m.dx_moe, torch.float16)
    full, more = R.lora(m.who.tolist(), ranks, scale, m.B, m.A, m.dy, torch.zeros(T, D), 22, torch.float16)
    R.check(m.dx, ref + full, bound + more + R.rounded(ref.abs() + full.abs() + bound + more, torch.float16), "dx")
    ra, ba, rb, bb = R.lora_grad(m.who.tolist(), ranks, scale, m.A, m.B, m.x, m.dy)
    R.check(m.dA, ra, ba, "dA")
    R.check(m.dB, rb, bb, "dB")


def test_layer_replayed_from_a_graph():
    """Other tokens, experts and adapters between the replays, and eager work of another layer on the way."""
    m, other = Layer(64, 2, seed=3), Layer(33, 2, seed=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.forward()
        m.backward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward()
        m.backward()
    for i in range(4):
        m.set_batch(20 + i)
        m.x.copy_(torch.randn(64, D, device="cuda"))
        m.dy.copy_(torch.randn(64, H, device="cuda"))
        for t in (m.xs, m.ys, m.dys, m.dxs):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        other.forward()
        torch.cuda.synchronize()
        got = m.results()
        for t in (m.xs, m.ys, m.dys, m.dxs, m.y, m.dx, m.dA, m.dB, m.dw):
            t.fill_(float("nan"))
        m.forward()
        m.backward()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, m.results())), i
