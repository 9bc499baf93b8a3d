"""The many-token operators next to the pruned-weight product: what is measured, and their plain forms.

Three operators that a program serving or fine-tuning pruned weights runs together:

  spmm   the MACKO-encoded projection applied to many tokens, for one weight or for one weight per expert
  lora   low-rank adapters of many requests added to a shared projection, and their weight gradients
  route  tokens sorted by expert (or by adapter) and back, with weights applied, and the gradients

`run` computes a case in its plain form, elementary torch operations in 32 bits, or, where `own` is set,
with the library's calls.  `exact` gives the same results from the definitions in 64 bits.
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
        # a small pruned layer and a handful of decoding requests: latency counts
        dict(name="spmm-2048-t5", op="spmm", rows=2048, cols=2048, groups=1, tok=5, sparsity=0.5, b=4, i8=False,
             y="f16"),
        # one decoding step of 32 requests through the pruned 12288 x 12288 weight at 70 %
        dict(name="spmm-12288-t32", op="spmm", rows=12288, cols=12288, groups=1, tok=32, sparsity=0.7, b=4, i8=False,
             y="f32"),
        # a prompt of 513 tokens through the same layer at 50 % with int8 values
        dict(name="spmm-12288-t513-i8", op="spmm", rows=12288, cols=12288, groups=1, tok=513, sparsity=0.5, b=4,
             i8=True, y="f16"),
        # eight pruned experts over tokens already sorted by expert, ragged groups, one of them empty
        dict(name="spmm-experts8-t257", op="spmm", rows=4096, cols=2048, groups=8, tok=257, sparsity=0.7, b=4,
             i8=False, y="f16"),
        # one request decoding with an adapter: the smallest call
        dict(name="lora-t1-r16", op="lora", tok=1, n_in=4096, n_out=4096, adapters=8, rank=16, x="f16", y="f32"),
        # a decoding batch of 61 requests over 40 adapters of mixed rank, some requests without one
        dict(name="lora-t61-r64", op="lora", tok=61, n_in=12288, n_out=12288, adapters=40, rank=64, x="f16",
             y="f32"),
        # prompts of a few requests, 4093 tokens in all
        dict(name="lora-t4093-r64", op="lora", tok=4093, n_in=4096, n_out=12288, adapters=6, rank=64, x="bf16",
             y="bf16"),
        # a fine-tuning micro-step of three small adapters, odd sizes
        dict(name="lora-grad-t300-r8", op="lora_grad", tok=300, n_in=1000, n_out=1504, adapters=3, rank=8, x="f16"),
        # a fine-tuning step over 8192 tokens of four adapters
        dict(name="lora-grad-t8192-r32", op="lora_grad", tok=8192, n_in=4096, n_out=4096, adapters=4, rank=32,
             x="bf16"),
        # a decoding batch through a router: sorted by expert, and back
        dict(name="route-t64-k2", op="route", tok=64, k=2, experts=8, dim=4096, x="bf16", grad=False),
        # odd sizes in fp32 with dropped choices, and the gradients
        dict(name="route-t1000-k3-f32", op="route", tok=1000, k=3, experts=13, dim=1111, x="f32", grad=True),
        # a training batch: there and back, and the gradients
        dict(name="route-t8191-k8", op="route", tok=8191, k=8, experts=64, dim=2048, x="bf16", grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer width: a multiple of 64 or of 8 mostly, any number now and then."""
    w = _log(rng, lo, hi)
    step = rng.choice([64, 64, 8, 1])
    return max(lo, w // step * step)


def draw(rng):
    op = rng.choice(["spmm", "spmm", "lora", "lora_grad", "route"])
    if op == "spmm":
        groups = rng.choice([1, 1, rng.randint(2, 8)])
        hi = 12288 if groups == 1 else 4096
        return dict(op=op, rows=_width(rng, 256, hi), cols=_width(rng, 256, hi), groups=groups, tok=_log(rng, 1, 500),
                    sparsity=round(rng.uniform(0.5, 0.92), 2), b=rng.choice([4, 4, 2, 8]), i8=rng.random() < 0.4,
                    y=rng.choice(["f16", "f32"]))
    if op == "lora":
        return dict(op=op, tok=_log(rng, 1, 4000), n_in=_width(rng, 256, 8192), n_out=_width(rng, 256, 8192),
                    adapters=_log(rng, 1, 48), rank=rng.choice([4, 8, 16, 24, 32, 64]), x=rng.choice(["f16", "bf16"]),
                    y=rng.choice(["x", "f32"]))
    if op == "lora_grad":
        return dict(op=op, tok=_log(rng, 16, 8000), n_in=_width(rng, 256, 4096), n_out=_width(rng, 256, 4096),
                    adapters=_log(rng, 1, 16), rank=rng.choice([4, 8, 16, 24, 32]), x=rng.choice(["f16", "bf16"]))
    return dict(op=op, tok=_log(rng, 1, 8000), k=rng.randint(1, 8), experts=_log(rng, 2, 200),
                dim=_width(rng, 256, 2048), x=rng.choice(["f16", "bf16", "f32"]), grad=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _macko_inputs(case, g, dev):
    """A random pruned weight (N(0, 0.02), uniform unstructured sparsity) in the MACKO layout of include/spmv.h."""
    n, k, b = case["rows"] * case["groups"], case["cols"], case["b"]
    rows, cols = (torch.rand(n, k, device=dev, generator=g) >= case["sparsity"]).nonzero(as_tuple=True)
    first = torch.ones(rows.numel(), dtype=torch.bool, device=dev)
    first[1:] = rows[1:] != rows[:-1]
    prev = torch.empty_like(cols)
    prev[1:] = cols[:-1]
    prev[first] = -1
    gap = cols - prev
    pads = (gap - 1) >> b                                  # entries that bridge a gap wider than 2^b
    code = (gap - 1 - (pads << b)).to(torch.uint8)
    length = torch.zeros(n, dtype=torch.int64, device=dev).index_add_(0, rows, pads + 1)
    align = 1024 // b
    start = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    start[1:] = torch.cumsum((length + align - 1) // align * align, 0)
    total = int(start[-1])
    run_ = torch.cumsum(pads + 1, 0)
    row_base = torch.cumsum(length, 0) - length
    pos = start[rows] + (run_ - 1 - row_base[rows])
    codes = torch.zeros(total, dtype=torch.uint8, device=dev)
    has = pads.nonzero().squeeze(1)
    rep = pads[has]
    at = torch.repeat_interleave(pos[has], rep)
    back = torch.arange(at.numel(), device=dev) - torch.repeat_interleave(torch.cumsum(rep, 0) - rep, rep)
    codes[at - 1 - back] = (1 << b) - 1
    codes[pos] = code
    vals = torch.zeros(total, dtype=torch.float16, device=dev)
    v = (torch.randn(pos.numel(), device=dev, generator=g) * 0.02).to(torch.float16)
    vals[pos] = torch.where(v == 0, torch.full_like(v, 0.02), v)
    per = 32 // b
    words = torch.zeros(total // per, dtype=torch.int32, device=dev)
    for i in range(per):
        words |= codes[i::per].to(torch.int32) << (b * i)
    s = dict(mrow_ptr=start.to(torch.int32), codes=words, vals=vals, scale=None)
    if case["i8"]:                                         # per row: scale max |v| / 127, values rounded to even
        row = torch.repeat_interleave(torch.arange(n, device=dev), start[1:] - start[:-1])
        top = torch.zeros(n, dtype=torch.float32, device=dev).index_reduce_(0, row, vals.float().abs(), "amax")
        s["scale"] = torch.where(top > 0, top / 127.0, torch.ones_like(top))
        s["vals"] = torch.round(vals.double() / s["scale"].double()[row]).clamp(-127, 127).to(torch.int8)
    return s


def _ragged(n, groups, g, dev):
    """Sorted-token offsets of `groups` ragged groups; the second one is empty where there are three or more."""
    w = torch.rand(groups, device=dev, generator=g) + 0.1
    if groups > 2:
        w[1] = 0
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * n + 0.5).to(torch.int32)
    cut[-1] = n
    return torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), cut])


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    randn = lambda *shape: torch.randn(*shape, device=dev, generator=g)  # noqa: E731
    s = {"case": case, "op": case["op"]}
    if case["op"] == "spmm":
        s.update(_macko_inputs(case, g, dev))
        s["x"] = randn(case["tok"], case["cols"]).to(torch.float16)
        s["offsets"] = _ragged(case["tok"], case["groups"], g, dev) if case["groups"] > 1 else None
        if own:                                            # laid out once for a weight, kept beside it
            import sparse_matrix_vector_amd as S
            s["m"] = S.MackoMatrix(case["rows"], case["cols"], s["mrow_ptr"], s["codes"], s["vals"], s["scale"],
                                   n_groups=case["groups"], bdelta=case["b"])
            s["ws"] = s["m"].workspace(case["tok"])
            s["out"] = torch.empty(case["tok"], case["rows"], dtype=DT[case["y"]], device=dev)
        return s
    if case["op"] in ("lora", "lora_grad"):
        dt, n, r, t = DT[case["x"]], case["adapters"], case["rank"], case["tok"]
        # requests come in runs of neighbouring tokens; about one in sixteen has no adapter (-1)
        runs = max(1, min(t, 4 * n))
        which = torch.randint(0, n, (runs,), device=dev, generator=g)
        none = torch.rand(runs, device=dev, generator=g) < 0.06
        if t > 1:
            which = torch.where(none, torch.full_like(which, -1), which)
        s["keys"] = which[torch.arange(t, device=dev) * runs // t].to(torch.int32)
        part = torch.randint(1, 5, (n,), device=dev, generator=g)
        s["ranks"] = torch.clamp(r * part // 4, min=1).to(torch.int32)
        s["scale"] = (torch.rand(n, device=dev, generator=g) + 0.5).float()
        s["A"] = (randn(n, r, case["n_in"]) / math.sqrt(case["n_in"])).to(dt)
        s["B"] = (randn(n, r, case["n_out"]) / math.sqrt(r)).to(dt)
        s["x"] = randn(t, case["n_in"]).to(dt)
        if case["op"] == "lora":
            ydt = dt if case["y"] == "x" else DT[case["y"]]
            s["base"] = randn(t, case["n_out"]).to(ydt)    # what the shared projection gave
        else:
            s["dy"] = randn(t, case["n_out"]).to(dt)
        if own:                                            # the batch's plan, shared by every layer's adapters
            import sparse_matrix_vector_amd as S
            s["plan"] = S.RoutePlan(t, 1, n).build(s["keys"])
            s["ws"] = torch.empty(S.lora_workspace_size(t, r), dtype=torch.uint8, device=dev)
            if case["op"] == "lora":
                s["out"] = torch.empty_like(s["base"])
            else:
                s["dA"] = torch.empty(s["A"].shape, dtype=torch.float32, device=dev)
                s["dB"] = torch.empty(s["B"].shape, dtype=torch.float32, device=dev)
        return s
    t, k, e, d, dt = case["tok"], case["k"], case["experts"], case["dim"], DT[case["x"]]
    # uneven experts (a router's popularity), distinct choices where there are enough experts, a few dropped (-1)
    pull = randn(e) + randn(t, e) * 1.5
    keys = torch.topk(pull, min(k, e), dim=1).indices
    keys = torch.cat([keys, keys[:, :1].expand(t, k - keys.shape[1])], 1) if keys.shape[1] < k else keys
    s["keys"] = torch.where(torch.rand(t, k, device=dev, generator=g) < 0.02, torch.full_like(keys, -1), keys)
    s["keys"] = s["keys"].to(torch.int32).contiguous()
    s["w"] = torch.softmax(randn(t, k), 1)
    s["x"] = randn(t, d).to(dt)
    s["ys"] = randn(t * k, d).to(dt)                       # what the experts gave, in sorted order
    s["xs"] = torch.zeros(t * k, d, dtype=dt, device=dev)  # rows past the last sorted one stay as they are
    if case["grad"]:
        s["dy"] = randn(t, d).to(dt)
        s["dxs"] = randn(t * k, d).to(dt)                  # what the experts' backward pass gave
        s["dys"] = torch.zeros(t * k, d, dtype=dt, device=dev)
    if own:
        import sparse_matrix_vector_amd as S
        s["plan"] = S.RoutePlan(t, k, e)
        s["y"] = torch.empty_like(s["x"])
        if case["grad"]:
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return {"spmm": _spmm, "lora": _lora, "lora_grad": _lora_grad, "route": _route}[s["op"]](s)


def _dense(s):
    """The weight, decoded to 32 bits: columns are the running sum of code + 1 in each row."""
    case, ptr, words = s["case"], s["mrow_ptr"].long(), s["codes"]
    n, k, b = ptr.numel() - 1, case["cols"], case["b"]
    shift = torch.arange(0, 32, b, device=words.device, dtype=torch.int32)
    step = ((words[:, None] >> shift) & ((1 << b) - 1)).reshape(-1).long() + 1
    row = torch.repeat_interleave(torch.arange(n, device=words.device), ptr[1:] - ptr[:-1])
    col = torch.cumsum(step, 0)
    col = col - (col - step)[torch.clamp(ptr[:-1], max=col.numel() - 1)][row] - 1
    w = torch.zeros(n, k + 1, device=words.device)
    w[row, torch.clamp(col, max=k)] = s["vals"].float() * (1.0 if s["scale"] is None else s["scale"][row])
    return w[:, :k]


def _spmm(s):
    case = s["case"]
    if own:
        return s["m"].apply(s["x"], s["out"], tok_offsets=s["offsets"], workspace=s["ws"])
    w, x = _dense(s), s["x"].float()
    if s["offsets"] is None:
        return (x @ w.t()).to(DT[case["y"]])
    # every expert for every token, then each token's own
    all_ = (x @ w.t()).view(case["tok"], case["groups"], case["rows"])
    mine = torch.searchsorted(s["offsets"], torch.arange(case["tok"], device=x.device, dtype=torch.int32),
                              right=True) - 1
    return all_[torch.arange(case["tok"], device=x.device), mine].to(DT[case["y"]])


def _mine(s):
    """[tok, adapters * rank]: the token's scale in the columns of its own adapter's rank, 0 elsewhere."""
    n, r = s["A"].shape[:2]
    a = torch.arange(n, device=s["x"].device)
    col = torch.arange(r, device=s["x"].device)
    m = (s["keys"][:, None, None] == a[None, :, None]) & (col[None, None, :] < s["ranks"][None, :, None])
    return (m * s["scale"][None, :, None]).reshape(-1, n * r)


def _lora(s):
    if own:
        import sparse_matrix_vector_amd as S
        p = s["plan"]
        return S.lora_apply(s["ranks"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"], s["base"],
                            s["out"], s["ws"])
    A, B = s["A"].float().flatten(0, 1), s["B"].float().flatten(0, 1)
    h = (s["x"].float() @ A.t()) * _mine(s)
    return (s["base"].float() + h @ B).to(s["base"].dtype)


def _lora_grad(s):
    if own:
        import sparse_matrix_vector_amd as S
        p = s["plan"]
        return S.lora_grad(s["ranks"], s["scale"], s["A"], s["B"], p.order, p.offsets, p.tiles, s["x"], s["dy"],
                           s["dA"], s["dB"], s["ws"])
    A, B, m = s["A"].float().flatten(0, 1), s["B"].float().flatten(0, 1), _mine(s)
    x, dy = s["x"].float(), s["dy"].float()
    return (((dy @ B.t()) * m).t() @ x).view(s["A"].shape), (((x @ A.t()) * m).t() @ dy).view(s["B"].shape)


def _route(s):
    case = s["case"]
    t, k, e = case["tok"], case["k"], case["experts"]
    if own:
        p = s["plan"].build(s["keys"])
        p.gather(s["x"], s["xs"])
        out = dict(offsets=p.offsets, order=p.order, pos=p.pos, xs=s["xs"], y=p.combine(s["ys"], s["y"], s["w"]))
        if case["grad"]:
            out["dys"], out["dw"] = p.combine_grad(s["dy"], s["ys"], s["w"], s["dys"], s["dw"])
            out["dx"] = p.combine(s["dxs"], s["dx"])
        return out
    key = s["keys"].reshape(-1).long()
    key = torch.where((key >= 0) & (key < e), key, torch.full_like(key, e))
    order = torch.sort(key, stable=True).indices           # dropped choices last
    kept = key < e
    pos = torch.empty_like(order)
    pos[order] = torch.arange(t * k, device=key.device)
    edges = torch.arange(e + 1, device=key.device)
    offsets = (key[None, :] < edges[:, None]).sum(1)
    live = kept[order]
    at = pos.view(t, k)
    w = torch.where(kept.view(t, k), s["w"], torch.zeros_like(s["w"]))
    xs = torch.where(live[:, None], s["x"][order // k], s["xs"])
    ys = torch.where(live[:, None], s["ys"], torch.zeros_like(s["ys"])).float()
    out = dict(offsets=offsets.int(), order=order.int(),
               pos=torch.where(kept, pos, torch.full_like(pos, -1)).int().view(t, k), xs=xs,
               y=(ys[at] * w[:, :, None]).sum(1).to(s["x"].dtype))
    if case["grad"]:
        dy = s["dy"].float()
        dys = (dy[order // k] * w.reshape(-1)[order][:, None]).to(s["x"].dtype)
        out["dys"] = torch.where(live[:, None], dys, s["dys"])
        out["dw"] = (ys[at] * dy[:, None, :]).sum(2)
        dxs = torch.where(live[:, None], s["dxs"], torch.zeros_like(s["dxs"])).float()
        out["dx"] = dxs[at].sum(1).to(s["x"].dtype)
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "spmm":
        n, k, t = case["rows"] * case["groups"], case["cols"], case["tok"]
        live = 1.0 - case["sparsity"]
        # stored entries: the live ones and those that bridge gaps wider than 2^b
        entries = n * k * live / (1.0 - case["sparsity"] ** (1 << case["b"]))
        nbytes = entries * ((1 if case["i8"] else 2) + case["b"] / 8) + 4 * (n + 1) + (4 * n if case["i8"] else 0)
        nbytes += t * k * 2 + t * case["rows"] * (4 if case["y"] == "f32" else 2)
        return {"bytes": nbytes, "flops": 2.0 * case["rows"] * k * live * t}
    if case["op"] in ("lora", "lora_grad"):
        t, r, n = case["tok"], case["rank"] * 0.625, case["adapters"]   # ranks are a quarter to the whole of it
        width = case["n_in"] + case["n_out"]
        # adapters that at least one of the batch's runs of tokens uses
        used = n * (1.0 - (1.0 - 1.0 / n) ** max(1, min(t, 4 * n)))
        if case["op"] == "lora":
            ysize = 4 if case["y"] == "f32" else 2
            return {"bytes": 2 * used * r * width + 2 * t * case["n_in"] + 2 * ysize * t * case["n_out"],
                    "flops": 2.0 * t * r * width}
        return {"bytes": 2 * used * r * width + 2 * t * width + 4 * n * case["rank"] * width,
                "flops": 4.0 * t * r * width}
    size = 4 if case["x"] == "f32" else 2
    t, slots, d = case["tok"], case["tok"] * case["k"], case["dim"]
    # x -> xs, ys -> y; with gradients dy, ys -> dys, dw and dxs -> dx; keys, weights, order and positions
    nbytes = size * d * (2 * t + 2 * slots) + 16 * slots
    flops = 2.0 * slots * d
    if case["grad"]:
        nbytes += size * d * (2 * t + 3 * slots) + 8 * slots
        flops += 4.0 * slots * d
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "spmm":
        n, cols, b = case["rows"] * case["groups"], case["cols"], case["b"]
        ptr = s["mrow_ptr"].cpu().numpy()
        bits = s["codes"].cpu().numpy().view(np.uint8)
        if b < 8:
            bits = np.stack([(bits >> (b * i)) & ((1 << b) - 1) for i in range(8 // b)], 1).reshape(-1)
        gaps, vals = torch.from_numpy(bits).cuda(), s["vals"].double()
        x = s["x"].double()
        cuts = [0, case["tok"]] if s["offsets"] is None else s["offsets"].tolist()
        y = torch.zeros(case["tok"], case["rows"], dtype=torch.float64, device="cuda")
        for g in range(case["groups"]):
            w = torch.zeros(case["rows"], cols + 1, dtype=torch.float64, device="cuda")
            for i in range(case["rows"]):
                lo, hi = int(ptr[g * case["rows"] + i]), int(ptr[g * case["rows"] + i + 1])
                c = torch.cumsum(gaps[lo:hi].int() + 1, 0) - 1
                w[i].index_copy_(0, c.clamp(max=cols), vals[lo:hi])
            if s["scale"] is not None:
                w *= s["scale"].double()[g * case["rows"]:(g + 1) * case["rows"], None]
            y[cuts[g]:cuts[g + 1]] = x[cuts[g]:cuts[g + 1]] @ w[:, :cols].t()
        return y
    if case["op"] in ("lora", "lora_grad"):
        keys, ranks = s["keys"].cpu(), s["ranks"].tolist()
        x = s["x"].double()
        if case["op"] == "lora":
            y = s["base"].double()
        else:
            dy = s["dy"].double()
            dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
            dB = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
        for a in range(case["adapters"]):
            at = (keys == a).nonzero().squeeze(1).cuda()
            A, B = s["A"][a, :ranks[a]].double(), s["B"][a, :ranks[a]].double()
            c = float(s["scale"][a])
            if case["op"] == "lora":
                y[at] += c * ((x[at] @ A.t()) @ B)
            else:
                dA[a, :ranks[a]] = c * ((dy[at] @ B.t()).t() @ x[at])
                dB[a, :ranks[a]] = c * ((x[at] @ A.t()).t() @ dy[at])
        return y if case["op"] == "lora" else (dA, dB)
    t, k, e, d = case["tok"], case["k"], case["experts"], case["dim"]
    keys = s["keys"].cpu().numpy().reshape(-1)
    order = np.concatenate([np.flatnonzero(keys == g) for g in range(e)])
    at = torch.from_numpy(order).cuda()
    x, w, ys = s["x"].double(), s["w"].double().reshape(-1), s["ys"].double()
    m = len(order)
    xs = s["xs"].double()
    xs[:m] = x[at // k]
    y = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    y.index_add_(0, at // k, ys[:m] * w[at, None])
    out = dict(offsets=None, order=None, pos=None, xs=xs, y=y)
    if case["grad"]:
        dy = s["dy"].double()
        out["dys"] = s["dys"].double()
        out["dys"][:m] = dy[at // k] * w[at, None]
        out["dw"] = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        out["dw"][at] = (ys[:m] * dy[at // k]).sum(1)
        out["dw"] = out["dw"].view(t, k)
        out["dx"] = torch.zeros(t, d, dtype=torch.float64, device="cuda")
        out["dx"].index_add_(0, at // k, s["dxs"].double()[:m])
    return out
