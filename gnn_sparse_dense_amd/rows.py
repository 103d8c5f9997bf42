"""Row operators: what a layer around the aggregation does with its rows when
each row belongs to one or more experts (or node types), the layer norm,
attention within segments, dropout and the loss of a linear classifier.

    route = RowRoute(expert, E)              # expert [T, k] int64: each row's experts
    xs = dispatch(route, x)                  # [T * k, N]: rows in expert order
    h = segment_matmul(xs, w, route.offsets) # w [E, N, O]: each expert's product
    out = combine(route, h, weight)          # [T, O]: summed back, weighted
    y = layer_norm(out, gamma, beta)

and, among the rows of each graph or sequence of a packed batch,

    a = segment_attention(q, k, v, offsets)  # q [R, H, D], k and v [K, Hk, D]
    y = dropout(a, 0.1, seed, 0, residual)   # no mask is stored

and the loss of a linear classifier over them, whose logits are not kept:

    loss = linear_cross_entropy(y, w, target)  # w [V, N], target int64 [R]

Rows are fp32, bf16 or fp16 matrices; sums are fp32 and outputs are rounded
once.  All run on torch's current stream of the tensors' device,
allocate through torch and never wait for the GPU, so they can be captured
into a graph (a backward pass only while no eager graph of the same leaves
lives that was built on the default stream, since torch ties a leaf's gradient
to the stream it was first used on: refused for every leaf that the pass leads
to from one of these operators).
All but RowRoute are differentiable (once);
the spmm_* functions are the C calls on the caller's tensors.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import HERE, SPMM_BF16, SPMM_F16, SPMM_F32, _check, _current_stream, _lib

if not os.path.exists(os.path.join(HERE, "_rows.so")):
    raise ImportError(f"{HERE}/_rows.so is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")

from . import _rows  # noqa: E402  (the autograd nodes, csrc/torch_rows.cpp)

_TYPES = {torch.float32: SPMM_F32, torch.bfloat16: SPMM_BF16, torch.float16: SPMM_F16}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_tensor(name, t, dtypes, shape, device):
    """t is what the library will read or write: it sees only the address."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d).replace('torch.', '') for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _check_rows_type(name, t, dim=2):
    if t.dim() != dim:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {dim}")
    if t.dtype not in _TYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return _TYPES[t.dtype]


@functools.lru_cache(maxsize=256)
def _workspace_bytes(call: str, *sizes: int) -> int:
    n = ctypes.c_int64()
    _check(getattr(_lib, call)(*sizes, ctypes.byref(n)))
    return n.value


def _workspace(device, call: str, *sizes: int):
    """(tensor or None, address, bytes) of one call's scratch memory."""
    n = _workspace_bytes(call, *sizes)
    if n == 0:
        return None, None, 0
    t = torch.empty(n, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), n


# ---------------------------------------------------------------- the C calls

def spmm_route_build(expert, E: int, offsets, order, position) -> None:
    """Sort the pairs of expert (int64, any shape) by expert into offsets
    int64 [E + 1], order and position int32 (expert's number of elements)."""
    pairs, E = expert.numel(), int(E)
    _check_tensor("expert", expert, (torch.int64,), expert.shape, offsets.device)
    _check_tensor("offsets", offsets, (torch.int64,), (E + 1,), offsets.device)
    _check_tensor("order", order, (torch.int32,), (pairs,), offsets.device)
    _check_tensor("position", position, (torch.int32,), expert.shape, offsets.device)
    ws, at, n = _workspace(offsets.device, "spmm_route_workspace", pairs, E)
    _check(_lib.spmm_route_build(_ptr(expert), pairs, E, _ptr(offsets), _ptr(order), _ptr(position), at, n,
                                 _current_stream(offsets)))


def _check_exchange(route, name, rows, count, weight):
    kind = _check_rows_type(name, rows)
    _check_tensor(name, rows, (rows.dtype,), (count, rows.shape[1]), route.device)
    if weight is None:
        return kind, kind
    _check_tensor("weight", weight, (torch.float32, rows.dtype), (route.T, route.k), route.device)
    return kind, _TYPES[weight.dtype]


def spmm_route_dispatch(route: "RowRoute", x, xs, weight=None) -> None:
    """xs [T * k, N] = rows of x [T, N] in expert order (times weight [T, k])."""
    kind, wkind = _check_exchange(route, "x", x, route.T, weight)
    _check_tensor("xs", xs, (x.dtype,), (route.T * route.k, x.shape[1]), route.device)
    _check(_lib.spmm_route_dispatch(_ptr(route.offsets), _ptr(route.order), route.T, route.k, route.E, _ptr(x),
                                    _ptr(weight), wkind, _ptr(xs), x.shape[1], kind, _current_stream(x)))


def spmm_route_combine(route: "RowRoute", rows, weight, out) -> None:
    """out [T, N] = the rows [T * k, N] summed back (weight [T, k] or None: 1)."""
    kind, wkind = _check_exchange(route, "rows", rows, route.T * route.k, weight)
    _check_tensor("out", out, (rows.dtype,), (route.T, rows.shape[1]), route.device)
    _check(_lib.spmm_route_combine(_ptr(route.offsets), _ptr(route.position), route.T, route.k, route.E, _ptr(rows),
                                   _ptr(weight), wkind, _ptr(out), rows.shape[1], kind, _current_stream(rows)))


def spmm_route_combine_backward(route: "RowRoute", rows, weight, dout, drows, dweight) -> None:
    """Gradients of combine: drows [T * k, N] and dweight [T, k], either may
    be None (rows too, without dweight)."""
    kind, wkind = _check_exchange(route, "dout", dout, route.T, weight)
    pairs = (route.T * route.k, dout.shape[1])
    if drows is not None:
        _check_tensor("drows", drows, (dout.dtype,), pairs, route.device)
    if dweight is not None:
        if rows is None:
            raise ValueError("rows are needed for dweight")
        _check_tensor("rows", rows, (dout.dtype,), pairs, route.device)
        types = (torch.float32, dout.dtype) if weight is None else (weight.dtype,)
        _check_tensor("dweight", dweight, types, (route.T, route.k), route.device)
        wkind = _TYPES[dweight.dtype]
    _check(_lib.spmm_route_combine_backward(_ptr(route.offsets), _ptr(route.order), route.T, route.k, route.E,
                                            _ptr(rows), _ptr(weight), wkind, _ptr(dout), _ptr(drows), _ptr(dweight),
                                            dout.shape[1], kind, _current_stream(dout)))


def _check_segment(rows_name, rows, width, dtype, offsets, R, E, device):
    _check_tensor(rows_name, rows, (dtype,), (R, width), device)
    _check_tensor("offsets", offsets, (torch.int64,), (E + 1,), device)


def spmm_segment_product(x, w, offsets, y) -> None:
    """y [R, O] = x [R, I] times w[e] [I, O] for the rows of each segment e."""
    kind = _check_rows_type("x", x)
    _check_rows_type("w", w, 3)
    E, I, O = w.shape
    _check_tensor("w", w, (x.dtype,), w.shape, x.device)
    _check_segment("x", x, I, x.dtype, offsets, x.shape[0], E, x.device)
    _check_tensor("y", y, (x.dtype,), (x.shape[0], O), x.device)
    _check(_lib.spmm_segment_product(_ptr(x), _ptr(w), _ptr(offsets), _ptr(y), x.shape[0], E, I, O, kind,
                                     _current_stream(x)))


def spmm_segment_product_dx(dy, w, offsets, dx) -> None:
    """dx [R, I] = dy [R, O] times the transpose of w[e] for each segment e."""
    kind = _check_rows_type("dy", dy)
    _check_rows_type("w", w, 3)
    E, I, O = w.shape
    _check_tensor("w", w, (dy.dtype,), w.shape, dy.device)
    _check_segment("dy", dy, O, dy.dtype, offsets, dy.shape[0], E, dy.device)
    _check_tensor("dx", dx, (dy.dtype,), (dy.shape[0], I), dy.device)
    _check(_lib.spmm_segment_product_dx(_ptr(dy), _ptr(w), _ptr(offsets), _ptr(dx), dy.shape[0], E, I, O, kind,
                                        _current_stream(dy)))


def spmm_segment_product_dw(x, dy, offsets, dw) -> None:
    """dw [E, I, O]: dw[e] = sum over the rows of segment e of x[r]^T dy[r]."""
    kind = _check_rows_type("x", x)
    _check_rows_type("dw", dw, 3)
    E, I, O = dw.shape
    _check_tensor("dw", dw, (x.dtype,), dw.shape, x.device)
    _check_segment("x", x, I, x.dtype, offsets, x.shape[0], E, x.device)
    _check_tensor("dy", dy, (x.dtype,), (x.shape[0], O), x.device)
    ws, at, n = _workspace(x.device, "spmm_segment_workspace", x.shape[0], E, I, O, kind)
    _check(_lib.spmm_segment_product_dw(_ptr(x), _ptr(dy), _ptr(offsets), _ptr(dw), x.shape[0], E, I, O, kind, at, n,
                                        _current_stream(x)))


def _check_norm(x, weight, bias):
    kind = _check_rows_type("x", x)
    wkind = kind
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check_tensor(name, t, (torch.float32, x.dtype), (x.shape[1],), x.device)
            wkind = _TYPES[t.dtype]
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"weight ({weight.dtype}) and bias ({bias.dtype}) must have one type")
    _check_tensor("x", x, (x.dtype,), x.shape, x.device)
    return kind, wkind


def spmm_layer_norm(x, weight, bias, y, mean=None, rstd=None, eps: float = 1e-5) -> None:
    """y = layer norm of each row of x [R, N]; mean and rstd (fp32 [R]) are
    what the backward pass reads."""
    kind, wkind = _check_norm(x, weight, bias)
    R, N = x.shape
    _check_tensor("y", y, (x.dtype,), x.shape, x.device)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _check_tensor(name, t, (torch.float32,), (R,), x.device)
    _check(_lib.spmm_layer_norm(_ptr(x), _ptr(weight), _ptr(bias), wkind, _ptr(y), _ptr(mean), _ptr(rstd), R, N,
                                float(eps), kind, _current_stream(x)))


def spmm_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias) -> None:
    """Gradients of the layer norm; any of dx [R, N], dweight and dbias [N]
    may be None."""
    kind, wkind = _check_norm(x, weight, None)
    R, N = x.shape
    _check_tensor("dy", dy, (x.dtype,), x.shape, x.device)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _check_tensor(name, t, (torch.float32,), (R,), x.device)
    if dx is not None:
        _check_tensor("dx", dx, (x.dtype,), x.shape, x.device)
    types = (torch.float32, x.dtype) if weight is None else (weight.dtype,)
    for name, t in (("dweight", dweight), ("dbias", dbias)):
        if t is not None:
            _check_tensor(name, t, types, (N,), x.device)
            wkind = _TYPES[t.dtype]
            types = (t.dtype,)
    ws, at, n = None, None, 0
    if dweight is not None or dbias is not None:
        ws, at, n = _workspace(x.device, "spmm_layer_norm_workspace", R, N, kind)
    _check(_lib.spmm_layer_norm_backward(_ptr(dy), _ptr(x), _ptr(weight), wkind, _ptr(mean), _ptr(rstd), _ptr(dx),
                                         _ptr(dweight), _ptr(dbias), R, N, kind, at, n, _current_stream(x)))


def _check_heads(q, k, v, offsets, key_offsets):
    kind = _check_rows_type("q", q, 3)
    _check_rows_type("k", k, 3)
    R, H, D = q.shape
    K, Hk = k.shape[:2]
    for name, t, shape in (("q", q, (R, H, D)), ("k", k, (K, Hk, D)), ("v", v, (K, Hk, D))):
        _check_tensor(name, t, (q.dtype,), shape, q.device)
    S = offsets.shape[0] - 1
    _check_tensor("offsets", offsets, (torch.int64,), (S + 1,), q.device)
    _check_tensor("key_offsets", key_offsets, (torch.int64,), (S + 1,), q.device)
    return (R, K, S, H, Hk, D), kind


def spmm_segment_attention(q, k, v, offsets, key_offsets, out, lse=None, causal: bool = False, scale: float = 1.0,
                           rest=None) -> None:
    """out [R, H, D] = attention of q [R, H, D] to k and v [K, Hk, D] within
    the segments; lse (fp32 [R, H]) and, of 16-bit rows, rest (as out: what its
    rounding leaves off) are what the backward pass reads."""
    sizes, kind = _check_heads(q, k, v, offsets, key_offsets)
    R, K, S, H, Hk, D = sizes
    _check_tensor("out", out, (q.dtype,), q.shape, q.device)
    if lse is not None:
        _check_tensor("lse", lse, (torch.float32,), (R, H), q.device)
    if rest is not None:
        _check_tensor("rest", rest, (q.dtype,), q.shape, q.device)
    ws, at, n = _workspace(q.device, "spmm_segment_attention_workspace", *sizes, kind)
    _check(_lib.spmm_segment_attention(_ptr(q), H * D, _ptr(k), Hk * D, _ptr(v), Hk * D, _ptr(offsets),
                                       _ptr(key_offsets), _ptr(out), _ptr(rest), _ptr(lse), *sizes, float(scale),
                                       int(causal), kind, at, n, _current_stream(q)))


def spmm_segment_attention_backward(q, k, v, offsets, key_offsets, out, lse, dout, dq, dk, dv, causal: bool = False,
                                    scale: float = 1.0, rest=None) -> None:
    """Gradients of the attention; any of dq [R, H, D], dk and dv [K, Hk, D]
    may be None."""
    sizes, kind = _check_heads(q, k, v, offsets, key_offsets)
    R, K, S, H, Hk, D = sizes
    _check_tensor("out", out, (q.dtype,), q.shape, q.device)
    _check_tensor("lse", lse, (torch.float32,), (R, H), q.device)
    _check_tensor("dout", dout, (q.dtype,), q.shape, q.device)
    if rest is not None:
        _check_tensor("rest", rest, (q.dtype,), q.shape, q.device)
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _check_tensor(name, t, (q.dtype,), like.shape, q.device)
    ws, at, n = _workspace(q.device, "spmm_segment_attention_backward_workspace", *sizes, kind)
    _check(_lib.spmm_segment_attention_backward(_ptr(q), H * D, _ptr(k), Hk * D, _ptr(v), Hk * D, _ptr(offsets),
                                                _ptr(key_offsets), _ptr(out), _ptr(rest), _ptr(lse), _ptr(dout),
                                                _ptr(dq), _ptr(dk), _ptr(dv), *sizes, float(scale), int(causal), kind,
                                                at, n, _current_stream(q)))


def spmm_dropout(x, residual, y, p: float, seed, offset: int = 0) -> None:
    """y = residual (or None: 0) + the kept elements of x / (1 - p); seed is
    int64 [1] on the GPU."""
    kind = _check_rows_type("x", x, x.dim())
    _check_tensor("x", x, (x.dtype,), x.shape, x.device)
    _check_tensor("y", y, (x.dtype,), x.shape, x.device)
    if residual is not None:
        _check_tensor("residual", residual, (x.dtype,), x.shape, x.device)
    _check_tensor("seed", seed, (torch.int64,), (1,), x.device)
    _check(_lib.spmm_dropout(_ptr(x), _ptr(residual), _ptr(y), x.numel(), float(p), _ptr(seed), int(offset), kind,
                             _current_stream(x)))


_REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}


@functools.lru_cache(maxsize=256)
def _loss_bytes(R: int, I: int, V: int, kind: int):
    """Bytes of the state and of the two workspaces."""
    n = [ctypes.c_int64() for _ in range(3)]
    _check(_lib.spmm_linear_cross_entropy_workspace(R, I, V, kind, *(ctypes.byref(b) for b in n)))
    return tuple(b.value for b in n)


def _check_loss(x, w, target, losses, name, reduction):
    kind = _check_rows_type("x", x)
    _check_rows_type("w", w)
    R, I = x.shape
    _check_tensor("x", x, (x.dtype,), x.shape, x.device)
    _check_tensor("w", w, (x.dtype,), (w.shape[0], I), x.device)
    _check_tensor("target", target, (torch.int64,), (R,), x.device)
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be 'none', 'sum' or 'mean', got {reduction!r}")
    _check_tensor(name, losses, (torch.float32,), (R,) if reduction == "none" else (), x.device)
    return (R, I, w.shape[0]), kind


def spmm_linear_cross_entropy(x, w, target, loss, reduction: str = "mean"):
    """loss (fp32, [R] for "none", else a scalar) of x [R, I] against the
    classes' rows w [V, I]; returns the state that the backward pass reads."""
    sizes, kind = _check_loss(x, w, target, loss, "loss", reduction)
    kept, n, _ = _loss_bytes(*sizes, kind)
    state = torch.empty(kept, dtype=torch.uint8, device=x.device)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _check(_lib.spmm_linear_cross_entropy(_ptr(x), _ptr(w), _ptr(target), _ptr(loss), *sizes, _REDUCTIONS[reduction],
                                          kind, _ptr(state), kept, _ptr(ws), n, _current_stream(x)))
    return state


def spmm_linear_cross_entropy_backward(x, w, target, dloss, dx, dw, state, reduction: str = "mean") -> None:
    """Gradients of the loss; either of dx [R, I] and dw [V, I] may be None."""
    sizes, kind = _check_loss(x, w, target, dloss, "dloss", reduction)
    kept, _, n = _loss_bytes(*sizes, kind)
    for name, t, like in (("dx", dx, x), ("dw", dw, w)):
        if t is not None:
            _check_tensor(name, t, (x.dtype,), like.shape, x.device)
    _check_tensor("state", state, (torch.uint8,), (kept,), x.device)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _check(_lib.spmm_linear_cross_entropy_backward(_ptr(x), _ptr(w), _ptr(target), _ptr(dloss), _ptr(dx), _ptr(dw),
                                                   *sizes, _REDUCTIONS[reduction], kind, _ptr(state), kept, _ptr(ws),
                                                   n, _current_stream(x)))


# ------------------------------------------------------- differentiable calls

class RowRoute:
    """Rows sorted by expert, built once per routing and applied many times.

    expert: int64 [T, k] (or [T]: one expert per row, such as a node's type)
    on the GPU; an id outside [0, num_experts) means no expert.  The pairs
    (row, choice) are sorted by expert, stably, those without an expert last:

    offsets : int64 [E + 1], places of each expert's pairs
    order   : int32 [T * k], the pair t * k + j at each place
    position: int32 [T, k], the place of each pair
    """

    __slots__ = ("offsets", "order", "position", "T", "k", "E")

    def __init__(self, expert, num_experts: int):
        self.E = int(num_experts)
        self.offsets, self.order, self.position, self.T, self.k = _rows.route_build(expert, self.E)

    @property
    def device(self):
        return self.offsets.device


def dispatch(route: RowRoute, x):
    """Rows of x [T, N] in expert order: [T * k, N], row route.position[t, j]
    = x[t]; rows from route.offsets[E] on (pairs without an expert) are zero.
    Differentiable in x."""
    return _rows.dispatch(route.offsets, route.order, route.position, route.T, route.k, route.E, x)


def combine(route: RowRoute, rows, weight=None):
    """out [T, N]: out[t] = sum over j of weight[t, j] * rows[position[t, j]],
    with rows [T * k, N] in expert order and weight [T, k] in fp32 or the
    rows' type (None: 1); pairs without an expert do not enter.
    Differentiable in rows and weight."""
    return _rows.combine(route.offsets, route.order, route.position, route.T, route.k, route.E, rows, weight)


def segment_matmul(x, w, offsets):
    """y [R, O]: y[r] = x[r] . w[e] for the rows offsets[e] <= r <
    offsets[e + 1] of x [R, I], with w [E, I, O] of x's type and offsets int64
    [E + 1] on the GPU (a RowRoute's, or the bounds of rows sorted by type);
    rows outside the segments are zero.  Differentiable in x and w."""
    return _rows.segment_matmul(x, w, offsets)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over the last dimension of x [..., N]: (x - mean) /
    sqrt(var + eps) * weight + bias with the biased variance; weight and bias
    [N] in fp32 or x's type (None: 1 and 0).  Differentiable in all three."""
    return _rows.layer_norm(x, weight, bias, eps)


def segment_attention(q, k, v, offsets, key_offsets=None, causal: bool = False, scale=None):
    """out [R, H, D]: each row of q [R, H, D] attends to the keys of its
    segment, the softmax of scale * q.k (None: D ** -0.5) times v, with k and v
    [K, Hk, D] of q's type, H a multiple of Hk (H / Hk heads share a key head)
    and D up to 128.  offsets int64 [S + 1] on the GPU bounds the segments'
    rows, as in segment_matmul; key_offsets theirs in k and v (None: offsets).
    causal: with n rows and m keys in a segment, its row i sees its keys
    j <= i + m - n, so a single new row sees all of its sequence.  Rows that see
    nothing, and rows outside the segments, are zero.  q, k and v may be parts
    of a wider row (a joint projection): they are read in place where their
    heads are packed.  Differentiable in q, k and v."""
    return _rows.segment_attention(q, k, v, offsets, key_offsets, causal, scale)


def dropout(x, p: float, seed, offset: int = 0, residual=None):
    """residual + x / (1 - p) where an element is kept (a share 1 - p of them),
    residual (None: 0) where it is dropped; x and residual of one shape (any)
    and type.  No mask is stored: seed (an int64 tensor of one element on the
    GPU, or a Python int), offset and an element's number in x say whether it
    is kept, forward and backward alike.  Give each step another seed (the
    tensor may change between the replays of a captured step, but not between
    a forward pass and its backward pass) and each call of a step another
    offset.  An int is copied to the GPU by each call (a launch more), and a
    captured call keeps it: every replay drops the same elements.
    Differentiable in x and residual (once)."""
    if not isinstance(seed, torch.Tensor):
        seed = torch.full((1,), int(seed), dtype=torch.int64, device=x.device)
    return _rows.dropout(x, p, seed, offset, residual)


def linear_cross_entropy(x, w, target, reduction: str = "mean"):
    """Softmax cross entropy of the logits x . w^T without keeping them, for
    x [R, I], a row of w [V, I] for each class and target int64 [R]: the loss
    of each row ("none", fp32 [R]), their "sum" or their "mean".  A target
    outside [0, V) means no class: the row has no loss, no gradient and does
    not count in the mean (which is zero over no rows).  Differentiable in x
    and w; in fp16 with "none", rows whose incoming gradient is below 2^-16 of
    the largest lose bits of theirs."""
    return _rows.linear_cross_entropy(x, w, target, reduction)
