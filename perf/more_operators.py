"""Operators of a quantised model's step: what is measured, and their plain forms.

Three operators next to the pruned and dense products, for weights held in 4 bits and for the table of token rows:

  q4     a projection of 4-bit weights with group scales applied to one token or many
  moe    a whole layer of 4-bit gated experts for the few tokens of a decoding step
  embed  the rows of a table of token embeddings, scaled, and the table's gradient

`run` computes a case in its plain form, elementary torch operations in 32 bits, or, where `own` is set,
with the library's calls.  `exact` gives the same results from the definitions in 64 bits.

4-bit weights, row by row: blocks of 128 columns (the last one filled up), each of sixteen 32-bit words.  Word
4 j + m of a block holds the columns 32 m + 8 j + e (e = 0 .. 7) of the block, column e in bits 4 i .. 4 i + 3 with
i = e / 2 + 4 (e % 2).  A group of 32, 64 or 128 columns has a scale and, where there are zero points, one of them:
weight = scale * (code - zero), with 8 for the zero point where there are none.
"""
import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoding request through a small projection: latency counts
        dict(name="q4-2048-t1", op="q4", rows=2048, cols=2048, tok=1, group=128, zeros=False, x="f16", y="x"),
        # one decoding request through the 12288 x 12288 projection
        dict(name="q4-12288-t1", op="q4", rows=12288, cols=12288, tok=1, group=128, zeros=False, x="f16", y="f32"),
        # seven requests, odd sizes, small groups with zero points
        dict(name="q4-5003x4100-t7", op="q4", rows=5003, cols=4100, tok=7, group=32, zeros=True, x="bf16", y="f32"),
        # a decoding batch of 48 requests
        dict(name="q4-12288-t48", op="q4", rows=12288, cols=12288, tok=48, group=64, zeros=True, x="bf16", y="x"),
        # a prompt of 513 tokens
        dict(name="q4-12288-t513", op="q4", rows=12288, cols=12288, tok=513, group=128, zeros=False, x="f16", y="x"),
        # one request through two of eight experts
        dict(name="moe-t1-e8-k2", op="moe", dim=2048, inter=4096, experts=8, k=2, tok=1, group=128, zeros=False,
             x="f16", y="x"),
        # a decoding batch of 16 requests over many small experts
        dict(name="moe-t16-e64-k8", op="moe", dim=2048, inter=1024, experts=64, k=8, tok=16, group=64, zeros=True,
             x="bf16", y="x"),
        # a large batch, odd widths
        dict(name="moe-t200-e24-k4", op="moe", dim=4096, inter=1500, experts=24, k=4, tok=200, group=128, zeros=False,
             x="f16", y="f32"),
        # the rows of a decoding batch
        dict(name="embed-t61", op="embed", vocab=50000, dim=4096, tok=61, x="bf16", y="x"),
        # the rows of a training batch
        dict(name="embed-t16384", op="embed", vocab=50000, dim=2048, tok=16384, x="f16", y="f32"),
        # the gradient of a small table in fp32, odd sizes
        dict(name="embed-grad-t1001", op="embed_grad", vocab=1003, dim=1111, tok=1001, x="f32", add=False),
        # the gradient of a training batch, some tokens far more common than others
        dict(name="embed-grad-t8191", op="embed_grad", vocab=50000, dim=2048, tok=8191, x="bf16", add=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer width: a multiple of 64 or of 8 mostly, any number now and then."""
    w = _log(rng, lo, hi)
    step = rng.choice([64, 64, 8, 1])
    return max(lo, w // step * step)


def draw(rng):
    op = rng.choice(["q4", "q4", "moe", "moe", "embed", "embed_grad"])
    if op == "q4":
        return dict(op=op, rows=_width(rng, 256, 12288), cols=_width(rng, 256, 12288), tok=_log(rng, 1, 500),
                    group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, x=rng.choice(["f16", "bf16"]),
                    y=rng.choice(["x", "f32"]))
    if op == "moe":
        dim, inter = _width(rng, 256, 4096), _width(rng, 128, 4096)
        experts = max(2, min(_log(rng, 4, 64), 400_000_000 // (3 * dim * inter)))
        return dict(op=op, dim=dim, inter=inter, experts=experts, k=rng.randint(1, min(8, experts)),
                    tok=_log(rng, 1, 200), group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                    x=rng.choice(["f16", "bf16"]), y=rng.choice(["x", "f32"]))
    vocab = _log(rng, 100, 50000)
    dim = _width(rng, 64, 2048)
    if op == "embed":
        return dict(op=op, vocab=vocab, dim=dim, tok=_log(rng, 1, 16384), x=rng.choice(["f16", "bf16", "f32"]),
                    y=rng.choice(["x", "f32"]))
    return dict(op=op, vocab=vocab, dim=dim, tok=_log(rng, 1, 8191), x=rng.choice(["f16", "bf16", "f32"]),
                add=rng.random() < 0.4)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _q4_inputs(rows, cols, case, g, dev):
    """(codes, scales, zeros) of random weights near N(0, 1 / cols): every group its own scale and, if there
    are any, its own zero point."""
    blocks = -(-cols // 128)
    zero = 8
    scales = (torch.rand(rows, blocks * 128 // case["group"], device=dev, generator=g) + 0.5) / (2.5 * math.sqrt(cols))
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(5, 11, scales.shape, device=dev, generator=g).to(torch.uint8)
    codes = torch.empty(rows, blocks * 16, dtype=torch.int32, device=dev)
    step = max(1, (1 << 25) // (blocks * 128))             # rows at a time
    for r in range(0, rows, step):
        n = min(step, rows - r)
        q = torch.randn(n, blocks * 128, device=dev, generator=g) * 2.5
        q = torch.clamp(torch.round(q) + zero, 0, 15).to(torch.int32).view(n, -1, 8)
        w = q[:, :, 0].clone()
        for i in range(1, 8):
            w |= q[:, :, i] << (4 * i)
        codes[r:r + n] = w
    return codes, scales.to(DT[case["x"]]), zeros


def _ids(case, g, dev):
    """Token ids whose frequency falls with the id, as in a text; about one in fifty is padding (-1)."""
    u = torch.rand(case["tok"], device=dev, generator=g, dtype=torch.float64)
    ids = torch.clamp(torch.exp(u * math.log(case["vocab"] + 1)).long() - 1, 0, case["vocab"] - 1)
    if case["tok"] > 1:
        ids = torch.where(torch.rand(case["tok"], device=dev, generator=g) < 0.02, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    randn = lambda *shape: torch.randn(*shape, device=dev, generator=g)  # noqa: E731
    s = {"case": case, "op": case["op"]}
    dt, t = DT[case["x"]], case["tok"]
    if own:
        import sparse_matrix_vector_amd as S
    if case["op"] == "q4":
        s["w"] = _q4_inputs(case["rows"], case["cols"], case, g, dev)
        s["x"] = randn(t, case["cols"]).to(dt)
        s["y"] = torch.empty(t, case["rows"], dtype=dt if case["y"] == "x" else DT[case["y"]], device=dev)
        if own:
            s["m"] = S.Q4Matrix(case["rows"], case["cols"], *s["w"], group=case["group"])
            s["ws"] = s["m"].workspace(t)
        return s
    if case["op"] == "moe":
        e, d, f, k = case["experts"], case["dim"], case["inter"], case["k"]
        # an expert's gate rows, then its up rows; all experts stacked
        s["gate_up"] = _q4_inputs(e * 2 * f, d, case, g, dev)
        s["down"] = _q4_inputs(e * d, f, case, g, dev)
        s["x"] = randn(t, d).to(dt)
        # a router's choices: uneven experts, distinct ones, a few dropped (-1)
        keys = torch.topk(randn(e) * 0.5 + randn(t, e), k, dim=1).indices
        if t > 1:
            keys = torch.where(torch.rand(t, k, device=dev, generator=g) < 0.02, torch.full_like(keys, -1), keys)
        s["keys"] = keys.to(torch.int32).contiguous()
        s["weights"] = torch.softmax(randn(t, k), 1)
        s["y"] = torch.empty(t, d, dtype=dt if case["y"] == "x" else DT[case["y"]], device=dev)
        if own:
            s["gu"] = S.Q4Matrix(2 * f, d, *s["gate_up"], group=case["group"], n_groups=e)
            s["dn"] = S.Q4Matrix(d, f, *s["down"], group=case["group"], n_groups=e)
            s["ws"] = torch.empty(S.moe_workspace_size(t, k, d, f), dtype=torch.uint8, device=dev)
        return s
    s["ids"] = _ids(case, g, dev)
    s["scale"] = math.sqrt(case["dim"])
    if case["op"] == "embed":
        s["table"] = (randn(case["vocab"], case["dim"]) * 0.02).to(dt)
        s["y"] = torch.empty(t, case["dim"], dtype=dt if case["y"] == "x" else DT[case["y"]], device=dev)
        return s
    s["dy"] = randn(t, case["dim"]).to(dt)
    # the gradient so far (of the steps before, or of the output layer that shares the table); overwritten without it
    s["dtable"] = randn(case["vocab"], case["dim"]) if case["add"] else torch.empty(case["vocab"], case["dim"], device=dev)
    s["first"] = s["dtable"].clone() if case["add"] else None
    if own:
        s["ws"] = torch.empty(S.embed_grad_workspace_size(t, case["vocab"], case["dim"]), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return {"q4": _q4, "moe": _moe, "embed": _embed, "embed_grad": _embed_grad}[s["op"]](s)


def _dense(w, cols, group, lo=0, hi=None):
    """Rows lo .. hi of the weight in 32 bits."""
    codes, scales, zeros = w
    codes = codes[lo:hi]
    n, blocks = codes.shape[0], codes.shape[1] // 16
    shift = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    q = ((codes.view(n, blocks, 4, 4, 1) >> shift) & 15).view(n, blocks, 4, 4, 2, 4)      # [.., j, m, odd, pair]
    q = q.permute(0, 1, 3, 2, 5, 4).reshape(n, -1, group).float()                        # [.., m, j, pair, odd]
    z = 8.0 if zeros is None else zeros[lo:hi].float()[:, :, None]
    return ((q - z) * scales[lo:hi].float()[:, :, None]).view(n, -1)[:, :cols]


def _q4(s):
    case = s["case"]
    if own:
        return s["m"].apply(s["x"], s["y"], workspace=s["ws"])
    return (s["x"].float() @ _dense(s["w"], case["cols"], case["group"]).t()).to(s["y"].dtype)


def _moe(s):
    case = s["case"]
    if own:
        import sparse_matrix_vector_amd as S
        return S.moe_apply(s["keys"], s["weights"], s["gu"], s["dn"], s["x"], s["y"], s["ws"])
    d, f, x = case["dim"], case["inter"], s["x"].float()
    y = torch.zeros(case["tok"], d, device=x.device)
    for e in range(case["experts"]):
        gu = x @ _dense(s["gate_up"], d, case["group"], e * 2 * f, (e + 1) * 2 * f).t()
        gate, up = gu[:, :f], gu[:, f:]
        out = (gate / (1.0 + torch.exp(-gate)) * up) @ _dense(s["down"], f, case["group"], e * d, (e + 1) * d).t()
        y += out * ((s["keys"] == e) * s["weights"]).sum(1)[:, None]
    return y.to(s["y"].dtype)


def _embed(s):
    if own:
        import sparse_matrix_vector_amd as S
        return S.embed_lookup(s["ids"], s["table"], s["y"], scale=s["scale"])
    ids = s["ids"].long()
    known = (ids >= 0) & (ids < s["case"]["vocab"])
    rows = s["table"][torch.where(known, ids, torch.zeros_like(ids))].float() * s["scale"]
    return torch.where(known[:, None], rows, torch.zeros_like(rows)).to(s["y"].dtype)


def _embed_grad(s):
    case = s["case"]
    if case["add"]:                                        # every pass adds to the same gradient
        s["dtable"].copy_(s["first"])
    if own:
        import sparse_matrix_vector_amd as S
        return S.embed_grad(s["ids"], s["dy"], s["dtable"], s["ws"], scale=s["scale"], accumulate=case["add"])
    ids, v, n = s["ids"].long(), case["vocab"], case["tok"]
    key = torch.where((ids >= 0) & (ids < v), ids, torch.full_like(ids, v))
    sorted_, order = torch.sort(key, stable=True)
    # sums over runs of equal ids, doubling their reach: a row adds the one `step` further if that has its id
    rows = s["dy"][order].float()
    step = 1
    while step < n:
        same = sorted_[step:] == sorted_[:-step]
        more = torch.where(same[:, None], rows[step:], torch.zeros_like(rows[step:]))
        rows = torch.cat([rows[:-step] + more, rows[-step:]])
        step *= 2
    first = torch.ones(n, dtype=torch.bool, device=ids.device)
    first[1:] = sorted_[1:] != sorted_[:-1]
    rows = rows * s["scale"]
    at = torch.where(first & (sorted_ < v), sorted_, torch.full_like(sorted_, v))
    out = torch.zeros(v + 1, case["dim"], device=ids.device)
    out[at] = rows
    if case["add"]:
        return s["dtable"].add_(out[:v])
    return s["dtable"].copy_(out[:v])


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def _q4_bytes(rows, cols, case):
    return rows * cols * (0.5 + (3.0 if case["zeros"] else 2.0) / case["group"])


def _distinct(case):
    """Expected number of distinct ids of a batch."""
    v = np.arange(case["vocab"], dtype=np.float64)
    p = (np.log(v + 2) - np.log(v + 1)) / math.log(case["vocab"] + 1)
    return float((1.0 - (1.0 - p) ** case["tok"]).sum())


def work(case):
    t, size = case["tok"], 4 if case["x"] == "f32" else 2
    if case["op"] == "q4":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": _q4_bytes(rows, cols, case) + t * cols * 2 + t * rows * (4 if case["y"] == "f32" else 2),
                "flops": 2.0 * t * rows * cols}
    if case["op"] == "moe":
        e, d, f, k = case["experts"], case["dim"], case["inter"], case["k"]
        used = e * (1.0 - (1.0 - k / e) ** t)              # experts that some token chooses
        nbytes = used * (_q4_bytes(2 * f, d, case) + _q4_bytes(d, f, case))
        return {"bytes": nbytes + t * d * (2 + (4 if case["y"] == "f32" else 2)) + 8 * t * k,
                "flops": 6.0 * t * k * d * f}
    if case["op"] == "embed":
        ysize = 4 if case["y"] == "f32" else size
        return {"bytes": case["dim"] * (_distinct(case) * size + t * ysize) + 4 * t, "flops": 1.0 * t * case["dim"]}
    # the gradient whole, or what it was and is where there are tokens (and all of it, set up for the pass)
    nbytes = case["dim"] * (t * size + 4 * case["vocab"]) + 4 * t
    if case["add"]:
        nbytes += 4 * case["dim"] * (case["vocab"] + 2 * _distinct(case))
    return {"bytes": nbytes, "flops": 1.0 * t * case["dim"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
_PLACE = [(e // 2) + 4 * (e % 2) for e in range(8)]        # nibble of column e of a word


def _dense64(w, cols, group, lo, hi):
    codes, scales, zeros = w
    c = codes[lo:hi].long() & 0xFFFFFFFF
    out = torch.empty(c.shape[0], c.shape[1] * 8, dtype=torch.float64, device=c.device)
    for word in range(16):
        j, m = divmod(word, 4)
        for e in range(8):
            out[:, 32 * m + 8 * j + e::128] = ((c[:, word::16] >> (4 * _PLACE[e])) & 15).double()
    rep = lambda a: torch.repeat_interleave(a[lo:hi].double(), group, dim=1)  # noqa: E731
    out -= 8.0 if zeros is None else rep(zeros)
    out *= rep(scales)
    return out[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "q4":
        x = s["x"].double()
        parts = [x @ _dense64(s["w"], case["cols"], case["group"], r, min(r + 2048, case["rows"])).t()
                 for r in range(0, case["rows"], 2048)]
        return torch.cat(parts, 1)
    if case["op"] == "moe":
        d, f, x = case["dim"], case["inter"], s["x"].double()
        y = torch.zeros(case["tok"], d, dtype=torch.float64, device=x.device)
        keys, w = s["keys"].cpu().tolist(), s["weights"].double().cpu()
        for e in range(case["experts"]):
            at = [(t, c) for t, row in enumerate(keys) for c, key in enumerate(row) if key == e]
            if not at:
                continue
            rows = torch.tensor([t for t, _ in at], device=x.device)
            share = torch.stack([w[t, c] for t, c in at]).to(x.device)
            gate = x[rows] @ _dense64(s["gate_up"], d, case["group"], e * 2 * f, e * 2 * f + f).t()
            up = x[rows] @ _dense64(s["gate_up"], d, case["group"], e * 2 * f + f, (e + 1) * 2 * f).t()
            h = gate * torch.sigmoid(gate) * up
            out = h @ _dense64(s["down"], f, case["group"], e * d, (e + 1) * d).t()
            y.index_add_(0, rows, out * share[:, None])
        return y
    ids = s["ids"].cpu().numpy()
    at = np.flatnonzero((ids >= 0) & (ids < case["vocab"]))
    rows, which = torch.from_numpy(at).cuda(), torch.from_numpy(ids[at].astype(np.int64)).cuda()
    if case["op"] == "embed":
        y = torch.zeros(case["tok"], case["dim"], dtype=torch.float64, device="cuda")
        y[rows] = s["scale"] * s["table"].double()[which]
        return y
    out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
    out.index_add_(0, which, s["scale"] * s["dy"].double()[rows])
    return out + s["first"].double() if case["add"] else out
