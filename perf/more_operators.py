"""Measured cases of attention within segments, dropout and the loss of a
linear classifier.

Three operators that a model on packed rows (the nodes of a batch of graphs,
the tokens of a batch of sequences) trains with, next to the aggregation, the
experts' products and the layer norm:

* attention: softmax(q k^T) v among the rows of each segment
  (segment_attention), and its three gradients; a single new row for each of
  many long sequences is one of its forms;
* dropout: elements kept by a counter-based generator, with the sum of a
  residual (dropout), and its gradients;
* loss: softmax cross entropy over the classes of a linear map, without the
  logits (linear_cross_entropy), and its two gradients.

`run` computes them in their plain form with elementary torch operations in
32 bits, or, where `own` is true, through the package.  `exact` restates the
definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of 32 sequences against their packed keys: one new row each
        dict(name="attention_step", op="attention", S=32, R=32, K=100003, pad=0, spread=0.9, H=32, G=4, D=128,
             type="bf16", causal=True, train=False),
        # a batch of small graphs, every node attends to its graph, fp32 as the aggregation
        dict(name="attention_graphs", op="attention", S=4096, R=100001, K=0, pad=0, spread=0.9, H=4, G=1, D=32,
             type="fp32", causal=False, train=True),
        # prompts of different lengths, packed, grouped heads, forward only
        dict(name="attention_prompt", op="attention", S=5, R=12001, K=0, pad=0, spread=0.8, H=32, G=4, D=128,
             type="bf16", causal=True, train=False),
        # a training batch of packed sequences
        dict(name="attention_train", op="attention", S=3, R=8192, K=0, pad=0, spread=0.4, H=16, G=4, D=128,
             type="bf16", causal=True, train=True),
        # rows that attend to another set of rows, odd lengths and an odd head, some rows behind the last segment
        dict(name="attention_cross", op="attention", S=9, R=3001, K=5003, pad=7, spread=0.7, H=6, G=1, D=72,
             type="fp16", causal=False, train=True),
        # one decoding step's block ends without dropout's gradient: latency only
        dict(name="dropout_step", op="dropout", R=32, N=2048, type="bf16", residual=True, p=0.1, train=False),
        # node features between two aggregation layers
        dict(name="dropout_nodes", op="dropout", R=1000000, N=64, type="fp32", residual=False, p=0.5, train=True),
        # a training batch of tokens, added to the residual stream
        dict(name="dropout_train", op="dropout", R=16381, N=4096, type="bf16", residual=True, p=0.1, train=True),
        # scoring a few continuations: the classes' rows are what is read
        dict(name="loss_step", op="loss", R=64, I=2048, V=32768, type="bf16", drop=0.0, reduction="none", train=False),
        # node classification, half of the nodes without a label, fp32
        dict(name="loss_nodes", op="loss", R=300007, I=128, V=47, type="fp32", drop=0.5, reduction="mean", train=True),
        # a training batch of tokens over a large vocabulary
        dict(name="loss_train", op="loss", R=8192, I=2048, V=65536, type="bf16", drop=0.05, reduction="mean",
             train=True),
        # odd sizes throughout, a gradient for each row
        dict(name="loss_ragged", op="loss", R=5003, I=1001, V=49999, type="fp16", drop=0.1, reduction="none",
             train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: any number one time in three, else a multiple of 16."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 1 / 3 else max(lo, n // 16 * 16)


def draw(rng):
    op = rng.choice(["attention", "attention", "dropout", "loss", "loss"])
    kind = rng.choice(["fp32", "bf16", "fp16"])
    train = rng.random() < 0.6
    if op == "attention":
        form = rng.choice(["step", "self", "self", "cross"])
        G, Hk = rng.choice([1, 1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        case = dict(op=op, pad=rng.choice([0, 0, 5]), spread=rng.uniform(0.0, 0.9), H=G * Hk, G=G,
                    D=rng.choice([16, 32, 40, 64, 64, 80, 96, 128, 128]), type=kind)
        if form == "step":
            S = _log(rng, 1, 128)
            return dict(S=S, R=S, K=S * _log(rng, 16, min(16384, (1 << 17) // S)), causal=True, train=False, **case)
        S = _log(rng, 1, 2048)
        # pairs of the longest segments, padded, are what the plain form holds
        top = (1 << 29 if kind != "fp32" else 1 << 27) // (S * case["H"])
        longest = max(2, int(math.sqrt(top)))
        mean = _log(rng, 1, max(2, min(4096, (1 << 15) // S + 16, int(longest / (1 + case["spread"])))))
        R = max(S, S * mean - rng.randrange(S))
        K = 0 if form == "self" else max(S, int(R * rng.choice([0.5, 1.0, 1.5])))
        return dict(S=S, R=R, K=K, causal=rng.random() < 0.5, train=train, **case)
    if op == "dropout":
        N = _width(rng, 8, 16384)
        return dict(op=op, R=_log(rng, 1, min(1000000, (1 << 26) // N)), N=N, type=kind, residual=rng.random() < 0.5,
                    p=rng.choice([0.0, 0.1, 0.1, 0.25, 0.5, 0.9]), train=train)
    I, V = _width(rng, 16, 2048), _width(rng, 2, 65536)
    top = (1 << 38) if kind != "fp32" else (1 << 36)
    return dict(op=op, R=_log(rng, 1, max(2, min(300007, (1 << 29) // V, top // (I * V)))), I=I, V=V, type=kind,
                drop=rng.choice([0.0, 0.1, 0.5]), reduction=rng.choice(["none", "mean", "sum"]), train=train)


def _spread(total, S, spread):
    """S lengths of `total` rows together, evenly spread from 1 - spread to 1 + spread of their mean."""
    at = [0]
    for i in range(S):
        share = 1 + spread * (2 * i / (S - 1) - 1) if S > 1 else 1
        at.append(at[-1] + share)
    ends = [int(round(total * a / at[-1])) for a in at]
    return [b - a for a, b in zip(ends, ends[1:])]


def _lengths(case):
    """Rows and keys of each segment."""
    rows = _spread(case["R"], case["S"], 0.0 if case["R"] == case["S"] else case["spread"])
    return rows, _spread(case["K"], case["S"], case["spread"]) if case["K"] else rows


def _pairs(case):
    """(query, key) pairs that meet, over all segments."""
    total = 0
    for n, m in zip(*_lengths(case)):
        if not case["causal"]:
            total += n * m
        else:                                          # query i sees keys up to i + m - n
            low = max(0, m - n + 1)
            total += (low + m) * (m - low + 1) // 2 if m else 0
    return total


def work(case):
    op, size = case["op"], BYTES[case["type"]]
    if op == "attention":
        rows, keys = case["R"], case["K"] or case["R"]
        per_q, per_k = case["H"] * case["D"] * size, case["H"] // case["G"] * case["D"] * size
        moved = 2 * (rows + case["pad"]) * per_q + 2 * keys * per_k + 16 * (case["S"] + 1)
        flops = 4 * _pairs(case) * case["H"] * case["D"]
        if case["train"]:
            # out and its gradient once more, dq, dk and dv
            moved += 2 * (rows + case["pad"]) * per_q + 2 * (keys + case["pad"]) * per_k
            flops *= 3
        return {"bytes": moved, "flops": flops}
    if op == "dropout":
        arrays = 2 + case["residual"] + (2 if case["train"] else 0)
        return {"bytes": arrays * case["R"] * case["N"] * size, "flops": 0}
    R, I, V = case["R"], case["I"], case["V"]
    kept = R * (1 - case["drop"])
    moved = size * (kept * I + V * I) + 8 * R + 4 * (R if case["reduction"] == "none" else 1)
    flops = 2 * kept * I * V
    if case["train"]:
        moved += size * (R * I + V * I)
        flops *= 3
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    op, kind, train = case["op"], TYPES[case["type"]], case["train"]
    s = dict(op=op, case=case, train=train)

    def normal(*shape, scale=1.0, grad=False):
        t = torch.randn(*shape, generator=g, device=DEVICE).mul_(scale).to(kind)
        return t.requires_grad_() if grad and train else t

    if op == "attention":
        rows, keys = _lengths(case)
        order = list(range(case["S"]))
        random.Random(seed).shuffle(order)
        rows, keys = [rows[i] for i in order], [keys[i] for i in order]
        H, Hk, D = case["H"], case["H"] // case["G"], case["D"]
        R = case["R"] + case["pad"]
        K = (case["K"] or case["R"]) + case["pad"]
        s["offsets"] = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int64, device=DEVICE)
        s["key_offsets"] = torch.tensor([0] + list(np.cumsum(keys)), dtype=torch.int64, device=DEVICE) if case["K"] else None
        s["longest"] = (max(rows), max(keys))           # the plain form pads to them
        s["q"] = normal(R, H, D, scale=1.5, grad=True)
        s["k"] = normal(K, Hk, D, grad=True)
        s["v"] = normal(K, Hk, D, grad=True)
        if train:
            s["dout"] = normal(R, H, D)
    elif op == "dropout":
        R, N = case["R"], case["N"]
        s["x"] = normal(R, N, grad=True)
        s["residual"] = normal(R, N, grad=True) if case["residual"] else None
        s["seed"] = torch.randint(-2 ** 62, 2 ** 62, (1,), generator=g, device=DEVICE)
        s["offset"] = 3                                 # which of a model's dropouts it is
        if train:
            s["dy"] = normal(R, N)
    else:
        R, I, V = case["R"], case["I"], case["V"]
        target = torch.randint(0, V, (R,), generator=g, device=DEVICE)
        s["w"] = normal(V, I, scale=I ** -0.5, grad=True)
        # rows that point somewhat towards their class
        x = torch.randn(R, I, generator=g, device=DEVICE) + 4.0 * s["w"].detach()[target].float()
        s["x"] = x.to(kind).requires_grad_() if train else x.to(kind)
        if case["drop"]:
            gone = torch.rand(R, generator=g, device=DEVICE) < case["drop"]
            target = torch.where(gone, torch.full_like(target, -1), target)
        s["target"] = target
        if train:
            s["dloss"] = torch.rand(R if case["reduction"] == "none" else (), generator=g, device=DEVICE) + 0.5
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        return {"attention": _own_attention, "dropout": _own_dropout, "loss": _own_loss}[op](s)
    with torch.no_grad():
        return {"attention": _plain_attention, "dropout": _plain_dropout, "loss": _plain_loss}[op](s)


def _own_attention(s):
    import gnn_sparse_dense_amd as G
    q, k, v = s["q"], s["k"], s["v"]
    out = G.segment_attention(q, k, v, s["offsets"], s["key_offsets"], causal=s["case"]["causal"])
    if not s["train"]:
        return {"out": out}
    dq, dk, dv = torch.autograd.grad(out, [q, k, v], s["dout"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _own_dropout(s):
    import gnn_sparse_dense_amd as G
    x, residual = s["x"], s["residual"]
    y = G.dropout(x, s["case"]["p"], s["seed"], s["offset"], residual)
    if not s["train"]:
        return {"y": y}
    if residual is None:
        return {"y": y, "dx": torch.autograd.grad(y, x, s["dy"])[0]}
    dx, dresidual = torch.autograd.grad(y, [x, residual], s["dy"])
    return {"y": y, "dx": dx, "dresidual": dresidual}


def _own_loss(s):
    import gnn_sparse_dense_amd as G
    loss = G.linear_cross_entropy(s["x"], s["w"], s["target"], s["case"]["reduction"])
    if not s["train"]:
        return {"loss": loss}
    dx, dw = torch.autograd.grad(loss, [s["x"], s["w"]], s["dloss"])
    return {"loss": loss, "dx": dx, "dw": dw}


def _slots(offsets, rows, longest):
    """Segment and place of each row in a padded batch; rows of no segment take the place `longest`."""
    S = offsets.numel() - 1
    row = torch.arange(rows, device=offsets.device)
    seg = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    live = (seg < S) & (row >= offsets[0])
    seg = seg.clamp(max=S - 1)
    return live, seg, torch.where(live, row - offsets[seg], torch.full_like(row, longest))


def _plain_attention(s):
    q, k, v = s["q"], s["k"], s["v"]
    kind, G, D = q.dtype, s["case"]["G"], s["case"]["D"]
    H, Hk = q.shape[1], k.shape[1]
    Lq, Lk = s["longest"]
    offsets = s["offsets"]
    key_offsets = offsets if s["key_offsets"] is None else s["key_offsets"]
    S = offsets.numel() - 1
    live, seg, slot = _slots(offsets, q.shape[0], Lq)
    klive, kseg, kslot = _slots(key_offsets, k.shape[0], Lk)
    zero = torch.zeros((), device=q.device)

    def padded(t, live, seg, slot, longest, heads):
        """[S * heads, longest, D] of the rows, zeros behind each segment's last."""
        p = torch.zeros(S, heads, longest + 1, D, device=q.device)
        p[seg, :, slot] = torch.where(live[:, None, None], t.float(), zero)
        return p[:, :, :longest].reshape(S * heads, longest, D)

    def packed(p, live, seg, slot, longest):
        rows = p.reshape(S, -1, longest, D)[seg, :, slot.clamp(max=longest - 1)]
        return torch.where(live[:, None, None], rows, zero).to(kind)

    # a group's query heads stand next to each other, so they share a key head's batch entry
    qp = padded(q, live, seg, slot, Lq, H).reshape(S * Hk, G * Lq, D)
    kp, vp = (padded(t, klive, kseg, kslot, Lk, Hk) for t in (k, v))
    n = offsets[1:] - offsets[:-1]
    m = key_offsets[1:] - key_offsets[:-1]
    i = torch.arange(Lq, device=q.device)
    j = torch.arange(Lk, device=q.device)
    seen = (i[None, :, None] < n[:, None, None]) & (j[None, None, :] < m[:, None, None])
    if s["case"]["causal"]:
        seen = seen & (j[None, None, :] <= i[None, :, None] + (m - n)[:, None, None])
    seen = seen[:, None, None]                          # [S, 1, 1, Lq, Lk]
    scale = D ** -0.5
    score = (torch.bmm(qp, kp.transpose(1, 2).contiguous()) * scale).view(S, Hk, G, Lq, Lk)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, zero, top))
    total = e.sum(-1, keepdim=True)
    p = (e / torch.where(total == 0, torch.ones_like(total), total)).view(S * Hk, G * Lq, Lk)
    out = torch.bmm(p, vp)
    result = {"out": packed(out, live, seg, slot, Lq)}
    if not s["train"]:
        return result
    dout = padded(s["dout"], live, seg, slot, Lq, H).reshape(S * Hk, G * Lq, D)
    dp = torch.bmm(dout, vp.transpose(1, 2).contiguous())
    ds = p * (dp - (dout * out).sum(-1, keepdim=True)) * scale
    result["dq"] = packed(torch.bmm(ds, kp), live, seg, slot, Lq)
    result["dk"] = packed(torch.bmm(ds.transpose(1, 2).contiguous(), qp), klive, kseg, kslot, Lk)
    result["dv"] = packed(torch.bmm(p.transpose(1, 2).contiguous(), dout), klive, kseg, kslot, Lk)
    return result


def _times(a, m):
    """High and low 32 bits of a * m, both below 2^32 and held in int64."""
    low, high = (a & 0xFFFF) * m, (a >> 16) * m
    return (high + (low >> 16)) >> 16, (low + ((high & 0xFFFF) << 16)) & 0xFFFFFFFF


def _plain_words(n, seed, offset):
    """32 random bits for each of n elements: Philox 4x32 with 10 rounds (Salmon et al. 2011), a counter for four."""
    at = torch.arange((n + 3) // 4, device=seed.device)
    a, b = at & 0xFFFFFFFF, at >> 32
    c, d = torch.full_like(at, offset & 0xFFFFFFFF), torch.full_like(at, offset >> 32 & 0xFFFFFFFF)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF
    for _ in range(10):
        ah, al = _times(a, 0xD2511F53)
        ch, cl = _times(c, 0xCD9E8D57)
        a, b, c, d = ch ^ b ^ k0, cl, ah ^ d ^ k1, al
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack([a, b, c, d], 1).reshape(-1)[:n]


def _plain_dropout(s):
    x, p = s["x"], s["case"]["p"]
    kept = (_plain_words(x.numel(), s["seed"], s["offset"]) >= round(p * 2 ** 32)).view(x.shape)
    scale = 1 / (1 - p) if p < 1 else 0.0
    zero = torch.zeros((), device=x.device)
    y = torch.where(kept, x.float() * scale, zero)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    result = {"y": y.to(x.dtype)}
    if s["train"]:
        result["dx"] = torch.where(kept, s["dy"].float() * scale, zero).to(x.dtype)
        if s["residual"] is not None:
            result["dresidual"] = s["dy"]
    return result


def _plain_loss(s):
    x, w, target, reduction = s["x"], s["w"], s["target"], s["case"]["reduction"]
    V = w.shape[0]
    live = (target >= 0) & (target < V)
    zero = torch.zeros((), device=x.device)
    xf, wf = torch.where(live[:, None], x.float(), zero), w.float()
    at = torch.where(live, target, torch.zeros_like(target))[:, None]
    logits = torch.mm(xf, wf.t())
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(1, keepdim=True)
    rows = (top + torch.log(total) - logits.gather(1, at))[:, 0]
    rows = torch.where(live, rows, zero)
    count = live.sum().clamp(min=1)
    loss = rows if reduction == "none" else rows.sum() / (count if reduction == "mean" else 1)
    if not s["train"]:
        return {"loss": loss}
    g = s["dloss"] / (count if reduction == "mean" else 1) * live
    p /= total
    p.scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float32))
    p *= g[:, None]
    return {"loss": loss, "dx": torch.mm(p, wf).to(x.dtype), "dw": torch.mm(p.t(), xf).to(w.dtype)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = {n: t.detach() if isinstance(t, torch.Tensor) else t for n, t in prepare(case, seed).items()}
    return {"attention": _exact_attention, "dropout": _exact_dropout, "loss": _exact_loss}[case["op"]](s)


def _exact_attention(s):
    """Segment by segment and, where gradients are asked for, by torch's own rules for them."""
    case = s["case"]
    if _pairs(case) * case["H"] * case["D"] > 1 << 42 or case["S"] > 5000:
        return None                                    # too long
    train, H, G, D = case["train"], case["H"], case["G"], case["D"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out = torch.zeros_like(q)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    rows = s["offsets"].tolist()
    keys = rows if s["key_offsets"] is None else s["key_offsets"].tolist()
    for a, b, c, d in zip(rows, rows[1:], keys, keys[1:]):
        if a == b or c == d:
            continue
        leaves = [t.transpose(0, 1).contiguous().requires_grad_(train) for t in (q[a:b], k[c:d], v[c:d])]
        qs, ks, vs = leaves
        score = torch.matmul(qs / math.sqrt(D), ks.repeat_interleave(G, 0).transpose(1, 2).contiguous())
        if case["causal"]:
            late = torch.ones(b - a, d - c, dtype=torch.bool, device=q.device).triu(d - c - (b - a) + 1)
            score = score.masked_fill(late, -1e300)
        weight = torch.softmax(score, 2)
        if case["causal"]:
            weight = weight * ~late                    # a query before the first key has no weights
        o = torch.matmul(weight, vs.repeat_interleave(G, 0))
        out[a:b] = o.detach().transpose(0, 1)
        if train:
            grads = torch.autograd.grad(o, leaves, s["dout"][a:b].double().transpose(0, 1).contiguous())
            dq[a:b], dk[c:d], dv[c:d] = (t.transpose(0, 1) for t in grads)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv} if train else {"out": out}


def _exact_dropout(s):
    """The generator on the host, in unsigned 64-bit words."""
    x, p = s["x"].double(), s["case"]["p"]
    n, mask = x.numel(), np.uint64(0xFFFFFFFF)
    key = int(s["seed"]) % 2 ** 64
    word = np.zeros(((n + 3) // 4, 4), dtype=np.uint64)
    word[:, 0] = np.arange(word.shape[0], dtype=np.uint64)
    word[:, 2] = s["offset"]
    for r in range(10):
        first, second = word[:, 0] * np.uint64(0xD2511F53), word[:, 2] * np.uint64(0xCD9E8D57)
        k0 = np.uint64((key + r * 0x9E3779B9) % 2 ** 32)
        k1 = np.uint64(((key >> 32) + r * 0xBB67AE85) % 2 ** 32)
        word[:, 0] = (second >> np.uint64(32)) ^ word[:, 1] ^ k0
        word[:, 2] = (first >> np.uint64(32)) ^ word[:, 3] ^ k1
        word[:, 1], word[:, 3] = second & mask, first & mask
    kept = torch.from_numpy(word.reshape(-1)[:n] >= np.uint64(round(p * 2 ** 32))).to(x.device).view(x.shape)
    factor = kept.double() / (1 - p)
    result = {"y": x * factor + (0 if s["residual"] is None else s["residual"].double())}
    if s["train"]:
        result["dx"] = s["dy"].double() * factor
        if s["residual"] is not None:
            result["dresidual"] = s["dy"].double()
    return result


def _exact_loss(s):
    """The labelled rows alone, with torch's own rules for the gradients."""
    w, target, train, reduction = s["w"].double(), s["target"], s["train"], s["case"]["reduction"]
    at = torch.nonzero((target >= 0) & (target < w.shape[0]))[:, 0]
    x = s["x"].double()[at].requires_grad_(train)
    w.requires_grad_(train)
    logp = torch.log_softmax(torch.mm(x, w.t()), 1)
    rows = -logp[torch.arange(at.numel(), device=x.device), target[at]]
    if reduction == "none":
        loss = torch.zeros(target.numel(), dtype=torch.float64, device=x.device).index_put((at,), rows)
    else:
        loss = rows.sum() / (max(1, at.numel()) if reduction == "mean" else 1)
    if not train:
        return {"loss": loss}
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device=x.device)
    dx[at], dw = torch.autograd.grad(loss, [x, w], s["dloss"].double())
    return {"loss": loss.detach(), "dx": dx, "dw": dw}
