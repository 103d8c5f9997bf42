"""Measured cases of the routed-row operators and of the layer norm.

Four operators that a mixture of experts (or a layer with typed nodes) runs
next to the neighbour aggregation:

* route: rows sorted by expert, stable (RowRoute);
* exchange: the route of a batch, its rows copied into expert order (dispatch)
  and the experts' rows summed back with weights (combine), and the gradients
  of both;
* segment: a product per expert over its run of rows (segment_matmul), and
  its two gradients;
* norm: layer norm over each row, and its three gradients.

`run` computes them in their plain form with elementary torch operations in
32 bits, or, where `own` is true, through the package.  `exact` restates the
definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-5


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a small batch: latency only
        dict(name="route_step", op="route", T=64, k=2, E=8, drop=0.0),
        # a training batch with many fine experts, some pairs over capacity
        dict(name="route_batch", op="route", T=131072, k=8, E=256, drop=0.02),
        # one decoding step through the experts' exchange, no gradients
        dict(name="exchange_step", op="exchange", T=48, k=2, E=16, N=1024, type="bf16", drop=0.0, train=False),
        # nodes of a graph, two experts each, narrow fp32 features
        dict(name="exchange_nodes", op="exchange", T=300007, k=2, E=11, N=64, type="fp32", drop=0.0, train=True),
        # a training batch of tokens, wide rows
        dict(name="exchange_train", op="exchange", T=16384, k=4, E=64, N=2048, type="bf16", drop=0.0, train=True),
        # bag-of-words features of an odd width, padded batch: a tenth of the pairs go nowhere
        dict(name="exchange_ragged", op="exchange", T=50021, k=3, E=24, N=1433, type="fp16", drop=0.1, train=True),
        # one decoding step: few rows, the experts' weights are what is read
        dict(name="segment_step", op="segment", R=96, E=16, I=1024, O=2048, type="bf16", drop=0.0, train=False),
        # nodes of seven types, each with its own linear map, fp32 as the aggregation
        dict(name="segment_types", op="segment", R=150001, E=7, I=128, O=256, type="fp32", drop=0.0, train=True),
        # a training batch through one layer of the experts
        dict(name="segment_train", op="segment", R=65536, E=32, I=1024, O=2048, type="bf16", drop=0.0, train=True),
        # one decoding step
        dict(name="norm_step", op="norm", R=32, N=2048, type="bf16", train=False),
        # node features between two aggregation layers
        dict(name="norm_nodes", op="norm", R=1000000, N=64, type="fp32", train=True),
        # a training batch of tokens
        dict(name="norm_train", op="norm", R=16381, N=4096, type="bf16", train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature width: any number one time in three, else a multiple of 16."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 1 / 3 else max(16, n // 16 * 16)


def draw(rng):
    op = rng.choice(["route", "exchange", "exchange", "segment", "segment", "norm", "norm"])
    if op == "route":
        k = rng.choice([1, 2, 4, 6, 8])
        E = max(k, _log(rng, 4, 512))
        return dict(op=op, T=_log(rng, 1, min(131072, (1 << 25) // E)), k=k, E=E, drop=rng.choice([0.0, 0.0, 0.05, 0.3]))
    kind = rng.choice(["fp32", "bf16", "fp16"])
    if op == "exchange":
        k = rng.choice([1, 2, 3, 4, 8])
        E = max(k, _log(rng, 4, 256))
        N = _width(rng, 16, 4096)
        most = min(300007, (1 << 27) // (N * k), (1 << 25) // E)
        return dict(op=op, T=_log(rng, 1, most), k=k, E=E, N=N, type=kind, drop=rng.choice([0.0, 0.0, 0.1]),
                    train=rng.random() < 0.6)
    if op == "segment":
        E = _log(rng, 1, 64)
        I, O = _width(rng, 16, 2048), _width(rng, 16, 2048)
        top = (1 << 37) if kind != "fp32" else (1 << 35)
        most = max(2, min(150001, top // (I * O)))
        return dict(op=op, R=_log(rng, 1, most), E=E, I=I, O=O, type=kind, drop=rng.choice([0.0, 0.0, 0.1]),
                    train=rng.random() < 0.6)
    N = _width(rng, 8, 16384)
    return dict(op=op, R=_log(rng, 1, min(1000000, (1 << 26) // N)), N=N, type=kind, train=rng.random() < 0.6)


def work(case):
    op = case["op"]
    if op == "route":
        R = case["T"] * case["k"]
        return {"bytes": 8 * R + 4 * R + 4 * R + 8 * (case["E"] + 1), "flops": 0}
    size = BYTES[case["type"]]
    if op == "exchange":
        T, R = case["T"], case["T"] * case["k"]
        kept = R * (1 - case["drop"])
        row = case["N"] * size
        moved = 16 * R + 8 * (case["E"] + 1) + T * row + R * row + kept * row + 4 * R + T * row
        flops = 2 * kept * case["N"]
        if case["train"]:
            moved += kept * row + T * row + T * row + R * row + 4 * R
            flops += 4 * kept * case["N"]
        return {"bytes": moved, "flops": flops}
    if op == "segment":
        R, I, O, E = case["R"], case["I"], case["O"], case["E"]
        kept = R * (1 - case["drop"])
        moved = size * (kept * I + R * O + E * I * O)
        flops = 2 * kept * I * O
        if case["train"]:
            moved += size * (kept * O + R * I + E * I * O)
            flops *= 3
        return {"bytes": moved, "flops": flops}
    R, N = case["R"], case["N"]
    if case["train"]:
        return {"bytes": size * (4 * R * N + 4 * N), "flops": 20 * R * N}
    return {"bytes": size * (2 * R * N + 2 * N), "flops": 8 * R * N}


# ---------------------------------------------------------------- the inputs

def _experts(case, g):
    """[T, k] int64: the k best of E uneven scores for each row; -1 for pairs that go nowhere."""
    T, k, E = case["T"], case["k"], case["E"]
    score = torch.randn(T, E, generator=g, device=DEVICE) + torch.randn(E, generator=g, device=DEVICE)
    best, expert = torch.topk(score, k, dim=1)
    if case["drop"]:
        gone = torch.rand(T, k, generator=g, device=DEVICE) < case["drop"]
        expert = torch.where(gone, torch.full_like(expert, -1), expert)
    return expert.contiguous(), torch.softmax(best, dim=1)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    op = case["op"]
    s = dict(op=op, case=case)
    if op == "route":
        s["expert"], _ = _experts(case, g)
        return s
    kind, train = TYPES[case["type"]], case["train"]
    s["train"] = train

    def normal(*shape, scale=1.0, shift=0.0, grad=False, dtype=kind):
        t = torch.randn(*shape, generator=g, device=DEVICE).mul_(scale).add_(shift).to(dtype)
        return t.requires_grad_() if grad and train else t

    if op == "exchange":
        T, k, N = case["T"], case["k"], case["N"]
        s["expert"], weight = _experts(case, g)
        s["weight"] = weight.requires_grad_() if train else weight
        s["x"] = normal(T, N, grad=True)
        s["y"] = normal(T * k, N, grad=True)          # what the experts return
        if train:
            s["dxs"], s["dout"] = normal(T * k, N), normal(T, N)
    elif op == "segment":
        R, E, I, O = case["R"], case["E"], case["I"], case["O"]
        share = torch.softmax(0.7 * torch.randn(E, generator=g, device=DEVICE), 0)
        share = torch.cat([share * (1 - case["drop"]), share.new_full((1,), case["drop"])])
        at = torch.multinomial(share, R, replacement=True, generator=g)
        rows = torch.bincount(at, minlength=E + 1)[:E]
        s["offsets"] = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
        s["longest"] = max(1, int(rows.max()))          # the plain form pads to it
        s["x"] = normal(R, I, grad=True)
        s["w"] = normal(E, I, O, scale=I ** -0.5, grad=True)
        if train:
            s["dy"] = normal(R, O)
    else:
        R, N = case["R"], case["N"]
        s["x"] = normal(R, N, scale=2.0, shift=0.5, grad=True)
        s["weight"] = normal(N, scale=0.1, shift=1.0, grad=True)
        s["bias"] = normal(N, scale=0.1, grad=True)
        if train:
            s["dy"] = normal(R, N)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        return {"route": _own_route, "exchange": _own_exchange, "segment": _own_segment, "norm": _own_norm}[op](s)
    with torch.no_grad():
        return {"route": _plain_route, "exchange": _plain_exchange, "segment": _plain_segment, "norm": _plain_norm}[op](s)


def _own_route(s):
    import gnn_sparse_dense_amd as G
    r = G.RowRoute(s["expert"], s["case"]["E"])
    return {"offsets": r.offsets, "order": r.order, "position": r.position}


def _own_exchange(s):
    import gnn_sparse_dense_amd as G
    r = G.RowRoute(s["expert"], s["case"]["E"])
    xs = G.dispatch(r, s["x"])
    out = G.combine(r, s["y"], s["weight"])
    if not s["train"]:
        return {"offsets": r.offsets, "xs": xs, "out": out}
    dx, dy, dweight = torch.autograd.grad([xs, out], [s["x"], s["y"], s["weight"]], [s["dxs"], s["dout"]])
    return {"offsets": r.offsets, "xs": xs, "out": out, "dx": dx, "dy": dy, "dweight": dweight}


def _own_segment(s):
    import gnn_sparse_dense_amd as G
    y = G.segment_matmul(s["x"], s["w"], s["offsets"])
    if not s["train"]:
        return {"y": y}
    dx, dw = torch.autograd.grad(y, [s["x"], s["w"]], s["dy"])
    return {"y": y, "dx": dx, "dw": dw}


def _own_norm(s):
    import gnn_sparse_dense_amd as G
    y = G.layer_norm(s["x"], s["weight"], s["bias"], EPS)
    if not s["train"]:
        return {"y": y}
    dx, dweight, dbias = torch.autograd.grad(y, [s["x"], s["weight"], s["bias"]], s["dy"])
    return {"y": y, "dx": dx, "dweight": dweight, "dbias": dbias}


def _plain_sort(expert, E):
    """offsets [E + 1], order and position: pairs in expert order, those without an expert last."""
    key = expert.reshape(-1)
    key = torch.where((key < 0) | (key >= E), torch.full_like(key, E), key)
    ranked, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ranked, torch.arange(E + 1, device=key.device))
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=key.device)
    return offsets, order, position.reshape(expert.shape)


def _plain_route(s):
    offsets, order, position = _plain_sort(s["expert"], s["case"]["E"])
    return {"offsets": offsets, "order": order.to(torch.int32), "position": position.to(torch.int32)}


def _plain_exchange(s):
    x, y, weight = s["x"], s["y"], s["weight"].float()
    kind = x.dtype
    offsets, order, position = _plain_sort(s["expert"], s["case"]["E"])
    T, k = position.shape
    kept = offsets[-1]
    live = (torch.arange(T * k, device=x.device) < kept)[:, None]
    there = (position < kept)[:, :, None]
    zero = torch.zeros((), device=x.device)
    xs = torch.where(live, x.float()[order // k], zero).to(kind)
    rows = torch.where(there, y.float()[position], zero)
    out = (weight[:, :, None] * rows).sum(1).to(kind)
    if not s["train"]:
        return {"offsets": offsets, "xs": xs, "out": out}
    dx = torch.where(there, s["dxs"].float()[position], zero).sum(1).to(kind)
    dout = s["dout"].float()
    dy = torch.where(live, weight.reshape(-1)[order][:, None] * dout[order // k], zero).to(kind)
    dweight = (rows * dout[:, None, :]).sum(2)
    return {"offsets": offsets, "xs": xs, "out": out, "dx": dx, "dy": dy, "dweight": dweight}


def _plain_segment(s):
    x, w, offsets = s["x"], s["w"].float(), s["offsets"]
    kind = x.dtype
    E, I, O = w.shape
    row = torch.arange(x.shape[0], device=x.device)
    seg = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    live = (seg < E)[:, None]
    seg = seg.clamp(max=E - 1)
    # rows of the last partial run past the end go to a slot of their own
    slot = torch.where(live[:, 0], row - offsets[seg], torch.full_like(row, s["longest"]))
    zero = torch.zeros((), device=x.device)

    def padded(t):
        p = torch.zeros(E, s["longest"] + 1, t.shape[1], device=t.device)
        p[seg, slot] = torch.where(live, t.float(), zero)
        return p

    xp = padded(x)
    y = torch.where(live, torch.bmm(xp, w)[seg, slot], zero).to(kind)
    if not s["train"]:
        return {"y": y}
    dyp = padded(s["dy"])
    dx = torch.where(live, torch.bmm(dyp, w.transpose(1, 2).contiguous())[seg, slot], zero).to(kind)
    dw = torch.bmm(xp.transpose(1, 2).contiguous(), dyp).to(s["w"].dtype)
    return {"y": y, "dx": dx, "dw": dw}


def _plain_norm(s):
    x, weight, bias = s["x"].float(), s["weight"].float(), s["bias"].float()
    kind = s["x"].dtype
    centred = x - x.mean(1, keepdim=True)
    rstd = torch.rsqrt((centred * centred).mean(1, keepdim=True) + EPS)
    unit = centred * rstd
    y = (unit * weight + bias).to(kind)
    if not s["train"]:
        return {"y": y}
    dy = s["dy"].float()
    g = dy * weight
    dx = (rstd * (g - g.mean(1, keepdim=True) - unit * (g * unit).mean(1, keepdim=True))).to(kind)
    return {"y": y, "dx": dx, "dweight": (dy * unit).sum(0).to(kind), "dbias": dy.sum(0).to(kind)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "route":
        return None                                    # whole numbers only
    s = {n: t.detach() if isinstance(t, torch.Tensor) else t for n, t in prepare(case, seed).items()}
    if op == "exchange":
        return _exact_exchange(s)
    if op == "segment":
        return _exact_segment(s)
    x, weight, bias = (s[n].double() for n in ("x", "weight", "bias"))
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    sd = torch.sqrt(var + EPS)
    out = {"y": (x - mean) / sd * weight + bias}
    if s["train"]:
        dy = s["dy"].double()
        N = x.shape[1]
        # y depends on x_j directly, through the mean and through the deviation
        direct = dy * weight / sd
        through_sd = (dy * weight * (x - mean)).sum(1, keepdim=True) / sd ** 3 / N
        out["dx"] = direct - direct.sum(1, keepdim=True) / N - (x - mean) * through_sd
        out["dweight"] = torch.einsum("rn,rn->n", dy, (x - mean) / sd)
        out["dbias"] = dy.sum(0)
    return out


def _exact_exchange(s):
    expert, E, x, y = s["expert"], s["case"]["E"], s["x"].double(), s["y"].double()
    T, k = expert.shape
    weight = s["weight"].double()
    where = torch.full((T * k,), -1, dtype=torch.int64, device=x.device)
    flat, at = expert.reshape(-1), 0
    for e in range(E):                                 # each expert takes its pairs in their order
        mine = torch.nonzero(flat == e)[:, 0]
        where[mine] = at + torch.arange(mine.numel(), device=x.device)
        at += mine.numel()
    xs, out = torch.zeros_like(y), torch.zeros_like(x)
    dx, dy, dweight = torch.zeros_like(x), torch.zeros_like(y), torch.zeros_like(weight)
    where = where.reshape(T, k)
    for j in range(k):
        t = torch.nonzero(where[:, j] >= 0)[:, 0]
        p = where[t, j]
        xs[p] = x[t]
        out[t] += weight[t, j, None] * y[p]
        if s["train"]:
            dout = s["dout"].double()[t]
            dx[t] += s["dxs"].double()[p]
            dy[p] = weight[t, j, None] * dout
            dweight[t, j] = (y[p] * dout).sum(1)
    got = {"offsets": None, "xs": xs, "out": out}
    return {**got, "dx": dx, "dy": dy, "dweight": dweight} if s["train"] else got


def _exact_segment(s):
    x, w, bounds = s["x"], s["w"], s["offsets"].tolist()
    E, I, O = w.shape
    y = torch.zeros(x.shape[0], O, dtype=torch.float64, device=x.device)
    dx = torch.zeros(x.shape[0], I, dtype=torch.float64, device=x.device)
    dw = torch.zeros(E, I, O, dtype=torch.float64, device=x.device)
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        xe, we = x[a:b].double(), w[e].double()
        y[a:b] = xe @ we
        if s["train"]:
            dye = s["dy"][a:b].double()
            dx[a:b] = dye @ we.t().contiguous()
            dw[e] = xe.t().contiguous() @ dye
    return {"y": y, "dx": dx, "dw": dw} if s["train"] else {"y": y}
