"""Python binding of the training-step operators of ``include/vcoll.h``: the
MoE router, the expert sort, the weighted combine (each with its gradient)
and the AdamW step.

As in the package itself, functions carry the C names and only marshal.
Per-rank buffers of one shape are given either as one contiguous tensor with
the ranks in front ([p, tokens, experts]) or as a sequence of p tensors
([tokens, experts]); results come in the form of the first argument that may
have either. Expert rows differ in number from rank to rank and are always a
sequence.
"""
from __future__ import annotations

import ctypes

from . import BF16, F32, MAX_RANKS, _check, _disjoint, _lib, _no_overlap, _on_current_gpu, _ptrs, _stream

ADAMW_GROUP = 128          # elements per scale of an 8-bit state


class _AdamwTensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("exp_avg_scale", ctypes.c_void_p), ("exp_avg_sq_scale", ctypes.c_void_p)]


class _AdamwHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


def _declare(lib) -> None:
    P, I, I64, VP = ctypes.POINTER, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
    lib.vcoll_moe_route.argtypes = [I, I64, I, I, I, I, P(VP), P(VP), P(VP), VP]
    lib.vcoll_moe_route_backward.argtypes = [I, I64, I, I, I, I, P(VP), P(VP), P(VP), P(VP), P(VP), VP]
    lib.vcoll_moe_sort.argtypes = [I, I64, I, I, P(VP), P(VP), VP, VP, I64, VP]
    lib.vcoll_moe_sort_workspace.argtypes = [I, I64, I, I, P(I64)]
    lib.vcoll_moe_combine_weighted.argtypes = [I, I64, I, I64, I, P(VP), P(I64), P(VP), P(VP), P(VP), VP]
    lib.vcoll_moe_combine_weighted_backward.argtypes = [I, I64, I, I64, I, P(VP), P(VP), P(I64), P(VP), P(VP), P(VP),
                                                        P(VP), VP]
    lib.vcoll_adamw.argtypes = [I, P(_AdamwTensor), I, I, I, P(_AdamwHyper), VP]
    lib.vcoll_adamw_unpack.argtypes = [I64, VP, VP, VP, VP, VP, VP, VP]
    for name in ("route", "route_backward", "sort", "sort_workspace", "combine_weighted", "combine_weighted_backward"):
        getattr(lib, "vcoll_moe_" + name).restype = I
    lib.vcoll_adamw.restype = I
    lib.vcoll_adamw_unpack.restype = I


_declare(_lib())


# -----------------------------------------------------------------------------
# per-rank buffers


def _first(x, what: str, name: str, dims: int):
    """(p, shape of one rank's buffer, dtype, device) of per-rank buffers in either form."""
    import torch
    if isinstance(x, torch.Tensor):
        p, shape, t = (x.shape[0] if x.dim() else 0), tuple(x.shape[1:]), x
    else:
        p = len(x)
        if p == 0 or not isinstance(x[0], torch.Tensor):
            raise ValueError(f"{what}: {name} must be a tensor or a sequence of tensors, one per rank")
        shape, t = tuple(x[0].shape), x[0]
    if not 1 <= p <= MAX_RANKS:
        raise ValueError(f"{what}: p={p} outside [1, {MAX_RANKS}]")
    if len(shape) != dims:
        raise ValueError(f"{what}: {name} must have {dims} dimensions per rank, got {tuple(shape)}")
    return p, shape, t.dtype, t.device


def _table(x, p: int, shape: tuple, dtype, dev, what: str, name: str):
    """(addresses of the p rank buffers, the tensors behind them) after the checks."""
    import torch
    if isinstance(x, torch.Tensor):
        if tuple(x.shape) != (p, *shape) or x.dtype is not dtype or x.device != dev or not x.is_contiguous():
            raise ValueError(f"{what}: {name} must be a contiguous {dtype} tensor {(p, *shape)} on {dev}, "
                             f"got {x.dtype} {tuple(x.shape)} on {x.device}")
        if x.numel() == 0:
            return (ctypes.c_void_p * p)(), []
        step = x.numel() // p * x.element_size()
        base = x.data_ptr()
        return (ctypes.c_void_p * p)(*range(base, base + p * step, step)), [x]
    ts = list(x)
    if len(ts) != p:
        raise ValueError(f"{what}: {name} must hold {p} rank buffers, got {len(ts)}")
    for t in ts:
        if tuple(t.shape) != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{what}: every {name} must be a contiguous {dtype} tensor {shape} on {dev}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return (ctypes.c_void_p * p)(*[t.data_ptr() if t.numel() else None for t in ts]), ts


def _new(like, p: int, shape: tuple, dtype, dev):
    """Rank buffers in the form of `like`."""
    import torch
    if isinstance(like, torch.Tensor):
        return torch.empty((p, *shape), dtype=dtype, device=dev)
    return [torch.empty(shape, dtype=dtype, device=dev) for _ in range(p)]


def _float_dtype(dtype, what: str) -> int:
    import torch
    if dtype is torch.float32:
        return F32
    if dtype is torch.bfloat16:
        return BF16
    raise TypeError(f"{what}: unsupported dtype {dtype}")


def _any(x):
    import torch
    return x if isinstance(x, torch.Tensor) else x[0]


# -----------------------------------------------------------------------------
# router


def vcoll_moe_route(logits, topk: int, normalise: bool = True, ids=None, weights=None):
    """Top-k experts and their softmax weights (see vcoll.h): logits [p,
    tokens, experts] float32 or bfloat16. Returns (ids [p, tokens, topk]
    int32, weights [p, tokens, topk] float32)."""
    import torch
    what = "vcoll_moe_route"
    p, (T, E), dt, dev = _first(logits, what, "logits", 2)
    code = _float_dtype(dt, what)
    if not 1 <= topk <= E:
        raise ValueError(f"{what}: topk={topk} outside [1, {E}]")
    z, zt = _table(logits, p, (T, E), dt, dev, what, "logits")
    _on_current_gpu(_any(logits))
    given = ids is not None or weights is not None
    ids = _new(logits, p, (T, topk), torch.int32, dev) if ids is None else ids
    weights = _new(logits, p, (T, topk), torch.float32, dev) if weights is None else weights
    i, it = _table(ids, p, (T, topk), torch.int32, dev, what, "ids")
    w, wt = _table(weights, p, (T, topk), torch.float32, dev, what, "weights")
    if given:
        _no_overlap(zt, it + wt, what)
        _disjoint(it + wt, what)
    _check(_lib().vcoll_moe_route(p, T, E, topk, code, int(bool(normalise)), z, i, w, _stream(_any(logits))), what)
    return ids, weights


def vcoll_moe_route_backward(logits, ids, weights, d_weights, normalise: bool = True, d_logits=None):
    """Gradient of vcoll_moe_route's weights (see vcoll.h): d_weights [p,
    tokens, topk] float32. Returns d_logits like logits."""
    import torch
    what = "vcoll_moe_route_backward"
    p, (T, E), dt, dev = _first(logits, what, "logits", 2)
    _, (_, K), _, _ = _first(ids, what, "ids", 2)
    code = _float_dtype(dt, what)
    if not 1 <= K <= E:
        raise ValueError(f"{what}: topk={K} outside [1, {E}]")
    z, zt = _table(logits, p, (T, E), dt, dev, what, "logits")
    i, it = _table(ids, p, (T, K), torch.int32, dev, what, "ids")
    w, wt = _table(weights, p, (T, K), torch.float32, dev, what, "weights")
    dw, dwt = _table(d_weights, p, (T, K), torch.float32, dev, what, "d_weights")
    _on_current_gpu(_any(logits))
    given = d_logits is not None
    d_logits = d_logits if given else _new(logits, p, (T, E), dt, dev)
    d, dtens = _table(d_logits, p, (T, E), dt, dev, what, "d_logits")
    if given:
        _no_overlap(zt + it + wt + dwt, dtens, what)
        _disjoint(dtens, what)
    _check(_lib().vcoll_moe_route_backward(p, T, E, K, code, int(bool(normalise)), z, i, w, dw, d,
                                           _stream(_any(logits))), what)
    return d_logits


# -----------------------------------------------------------------------------
# expert sort


def vcoll_moe_sort_workspace(p: int, tokens: int, topk: int, experts_per_rank: int) -> int:
    """Bytes of device workspace that vcoll_moe_sort needs for these sizes."""
    n = ctypes.c_int64()
    _check(_lib().vcoll_moe_sort_workspace(p, tokens, topk, experts_per_rank, ctypes.byref(n)),
           "vcoll_moe_sort_workspace")
    return n.value


def vcoll_moe_sort(ids, experts_per_rank: int, slots=None, offsets=None, workspace=None):
    """Token rows sorted by expert, on the device (see vcoll.h): ids [p,
    tokens, topk] int32. Returns (slots [p, tokens*topk, 2] int32 for
    vcoll_moe_dispatch and the combines, offsets [p, experts_per_rank + 1]
    int32). The workspace is made when None."""
    import torch
    what = "vcoll_moe_sort"
    p, (T, K), dt, dev = _first(ids, what, "ids", 2)
    if experts_per_rank < 1:
        raise ValueError(f"{what}: experts_per_rank={experts_per_rank} must be positive")
    i, it = _table(ids, p, (T, K), torch.int32, dev, what, "ids")
    _on_current_gpu(_any(ids))
    given = slots is not None or offsets is not None or workspace is not None
    slots = _new(ids, p, (T * K, 2), torch.int32, dev) if slots is None else slots
    offsets = torch.empty((p, experts_per_rank + 1), dtype=torch.int32, device=dev) if offsets is None else offsets
    s, st = _table(slots, p, (T * K, 2), torch.int32, dev, what, "slots")
    if tuple(offsets.shape) != (p, experts_per_rank + 1) or offsets.dtype is not torch.int32 or \
            offsets.device != dev or not offsets.is_contiguous():
        raise ValueError(f"{what}: offsets must be a contiguous int32 tensor {(p, experts_per_rank + 1)} on {dev}")
    if workspace is None:
        need = vcoll_moe_sort_workspace(p, T, K, experts_per_rank)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"{what}: workspace must be a contiguous tensor on {dev}")
    size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if given:
        out = st + [offsets] + ([workspace] if size else [])
        _no_overlap(it, out, what)
        _disjoint(out, what)
    _check(_lib().vcoll_moe_sort(p, T, K, experts_per_rank, i, s, offsets.data_ptr(),
                                 workspace.data_ptr() if size else None, size, _stream(_any(ids))), what)
    return slots, offsets


# -----------------------------------------------------------------------------
# weighted combine


def _expert_rows(expert, p: int, hidden, dtype, dev, what: str, name: str):
    """(addresses, row counts, the tensors) of p buffers [rows_j, hidden]."""
    ts = list(expert)
    if len(ts) != p:
        raise ValueError(f"{what}: {name} must hold {p} rank buffers, got {len(ts)}")
    for t in ts:
        if t.dim() != 2 or t.shape[1] != hidden or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{what}: every {name} must be a contiguous {dtype} tensor [rows, {hidden}] on {dev}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return _ptrs(ts), (ctypes.c_int64 * p)(*[t.shape[0] for t in ts]), ts


def vcoll_moe_combine_weighted(expert_out, slots, weights, tokens: int, topk: int, out=None):
    """Weighted sum of every token's expert rows (see vcoll.h): expert_out p
    tensors [rows_j, hidden]; slots [p, tokens*topk, 2] int32 of the dispatch;
    weights [p, tokens, topk] float32, or None for ones (the gradient of the
    dispatch). Returns out [p, tokens, hidden], in the form of slots."""
    import torch
    what = "vcoll_moe_combine_weighted"
    p, _, _, dev = _first(slots, what, "slots", 2)
    T, K = int(tokens), int(topk)
    first = expert_out[0]
    if first.dim() != 2:
        raise ValueError(f"{what}: expert_out must be [rows, hidden] per rank")
    H, dt = first.shape[1], first.dtype
    code = _float_dtype(dt, what)
    s, st = _table(slots, p, (T * K, 2), torch.int32, dev, what, "slots")
    w, wt = (None, []) if weights is None else _table(weights, p, (T, K), torch.float32, dev, what, "weights")
    _on_current_gpu(_any(slots))
    e, rows, et = _expert_rows(expert_out, p, H, dt, dev, what, "expert_out")
    given = out is not None
    out = out if given else _new(slots, p, (T, H), dt, dev)
    o, ot = _table(out, p, (T, H), dt, dev, what, "out")
    if given:
        _no_overlap(et + st + wt, ot, what)
        _disjoint(ot, what)
    _check(_lib().vcoll_moe_combine_weighted(p, T, K, H, code, e, rows, s, w, o, _stream(_any(slots))), what)
    return out


def vcoll_moe_combine_weighted_backward(d_out, expert_out, slots, weights, topk: int, d_expert_out=None,
                                        d_weights=None):
    """Gradients of vcoll_moe_combine_weighted (see vcoll.h): d_out [p,
    tokens, hidden]. Returns (d_expert_out, p tensors like expert_out;
    d_weights [p, tokens, topk] float32). Rows that no slot names are left as
    they are in a given d_expert_out and zero in one made here."""
    import torch
    what = "vcoll_moe_combine_weighted_backward"
    p, (T, H), dt, dev = _first(d_out, what, "d_out", 2)
    K = int(topk)
    code = _float_dtype(dt, what)
    g, gt = _table(d_out, p, (T, H), dt, dev, what, "d_out")
    s, st = _table(slots, p, (T * K, 2), torch.int32, dev, what, "slots")
    w, wt = _table(weights, p, (T, K), torch.float32, dev, what, "weights")
    _on_current_gpu(_any(d_out))
    e, rows, et = _expert_rows(expert_out, p, H, dt, dev, what, "expert_out")
    given = d_expert_out is not None or d_weights is not None
    if d_expert_out is None:
        d_expert_out = [torch.zeros_like(t) for t in et]
    de, drows, det = _expert_rows(d_expert_out, p, H, dt, dev, what, "d_expert_out")
    if list(drows) != list(rows):
        raise ValueError(f"{what}: d_expert_out must have the rows of expert_out")
    d_weights = _new(d_out, p, (T, K), torch.float32, dev) if d_weights is None else d_weights
    dw, dwt = _table(d_weights, p, (T, K), torch.float32, dev, what, "d_weights")
    if given:
        _no_overlap(gt + st + wt + et, det + dwt, what)
        _disjoint(det + dwt, what)
    _check(_lib().vcoll_moe_combine_weighted_backward(p, T, K, H, code, g, e, rows, s, w, de, dw,
                                                      _stream(_any(d_out))), what)
    return d_expert_out, d_weights


# -----------------------------------------------------------------------------
# AdamW


def adamw_state(params, bits: int = 32):
    """Zero states for vcoll_adamw, as its keyword arguments: exp_avg and
    exp_avg_sq (float32, or 8-bit codes with their scales) and, for bfloat16
    parameters, the float32 master copies."""
    import torch
    if bits not in (32, 8):
        raise ValueError(f"adamw_state: bits={bits} must be 32 or 8")
    ps = list(params)
    kind = torch.float32 if bits == 32 else torch.uint8
    state = {n: [torch.zeros(t.shape, dtype=kind, device=t.device) for t in ps] for n in ("exp_avg", "exp_avg_sq")}
    if bits == 8:
        for n in ("exp_avg_scale", "exp_avg_sq_scale"):
            state[n] = [torch.ones(-(-t.numel() // ADAMW_GROUP), device=t.device) for t in ps]
    if ps and ps[0].dtype is torch.bfloat16:
        state["master"] = [t.float() for t in ps]
    return state


class AdamwStep:
    """An AdamW step over tensors that were checked and marshalled once; each
    call enqueues one step on torch's current stream, in place."""

    def __init__(self, table, count: int, codes: tuple, keep: list):
        self._table, self._count, self._codes, self._keep = table, count, codes, keep

    def __call__(self, *, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.01, grad_scale: float = 1.0, seed: int = 0) -> None:
        if self._count == 0:
            return
        _on_current_gpu(self._keep[0])
        hyper = _AdamwHyper(lr, beta1, beta2, eps, weight_decay, grad_scale, step, seed & 0xFFFFFFFF, 0)
        _check(_lib().vcoll_adamw(self._count, self._table, *self._codes, ctypes.byref(hyper),
                                  _stream(self._keep[0])), "vcoll_adamw")


def prepare_adamw(params, grads, exp_avg, exp_avg_sq, master=None, exp_avg_scale=None,
                  exp_avg_sq_scale=None) -> AdamwStep:
    """Checks the tensors of an AdamW step (see vcoll.h) and returns it; it
    does not run. params float32 or bfloat16 (then with float32 master
    copies), grads float32 or bfloat16, exp_avg and exp_avg_sq float32 or
    uint8 codes (then with float32 scales, one per 128 elements)."""
    import torch
    what = "vcoll_adamw"
    ps = list(params)
    if not ps:
        return AdamwStep(None, 0, (F32, F32, 32), [])
    sides = [("params", ps), ("grads", list(grads)), ("exp_avg", list(exp_avg)), ("exp_avg_sq", list(exp_avg_sq))]
    dev = ps[0].device
    pcode = _float_dtype(ps[0].dtype, what)
    gcode = _float_dtype(sides[1][1][0].dtype, what) if sides[1][1] else F32
    if not sides[2][1] or sides[2][1][0].dtype not in (torch.float32, torch.uint8):
        raise TypeError(f"{what}: exp_avg must be float32 or uint8 tensors")
    kind = sides[2][1][0].dtype
    bits = 32 if kind is torch.float32 else 8
    if (pcode == BF16) != (master is not None):
        raise ValueError(f"{what}: bfloat16 parameters need float32 master copies, float32 ones take none")
    if (bits == 8) != (exp_avg_scale is not None) or (bits == 8) != (exp_avg_sq_scale is not None):
        raise ValueError(f"{what}: 8-bit states need both scales, float32 ones take none")
    if master is not None:
        sides.append(("master", list(master)))
    scales = [] if bits == 32 else [("exp_avg_scale", list(exp_avg_scale)),
                                    ("exp_avg_sq_scale", list(exp_avg_sq_scale))]
    dtypes = {"params": ps[0].dtype, "grads": torch.bfloat16 if gcode == BF16 else torch.float32, "exp_avg": kind,
              "exp_avg_sq": kind, "master": torch.float32}
    for name, ts in sides + scales:
        if len(ts) != len(ps):
            raise ValueError(f"{what}: {len(ps)} params but {len(ts)} {name}")
        for k, t in enumerate(ts):
            n = ps[k].numel()
            want = n if name in dtypes else -(-n // ADAMW_GROUP)
            if t.numel() != want or t.dtype is not dtypes.get(name, torch.float32) or t.device != dev or \
                    not t.is_contiguous():
                raise ValueError(f"{what}: {name}[{k}] must be a contiguous {dtypes.get(name, torch.float32)} tensor "
                                 f"of {want} elements on {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    _on_current_gpu(ps[0])
    written = [t for name, ts in sides + scales if name != "grads" for t in ts]
    _disjoint(written, what)
    _no_overlap(sides[1][1], written, what)
    columns = dict(sides + scales)
    table = (_AdamwTensor * len(ps))()
    fields = dict(param="params", grad="grads", master="master", exp_avg="exp_avg", exp_avg_sq="exp_avg_sq",
                  exp_avg_scale="exp_avg_scale", exp_avg_sq_scale="exp_avg_sq_scale")
    for k, row in enumerate(table):
        row.n = ps[k].numel()
        for field, column in fields.items():
            if column in columns and row.n:
                setattr(row, field, columns[column][k].data_ptr())
    return AdamwStep(table, len(ps), (pcode, gcode, bits), ps + [t for ts in columns.values() for t in ts])


def vcoll_adamw(params, grads, exp_avg, exp_avg_sq, *, lr: float, step: int, master=None, exp_avg_scale=None,
                exp_avg_sq_scale=None, **hyper) -> None:
    """One AdamW step over many tensors, in place (see prepare_adamw for the
    tensors, AdamwStep for the numbers). A program that keeps its tensors
    prepares the step once instead."""
    prepare_adamw(params, grads, exp_avg, exp_avg_sq, master, exp_avg_scale, exp_avg_sq_scale)(lr=lr, step=step,
                                                                                            **hyper)


def vcoll_adamw_unpack(exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, exp_avg_out=None, exp_avg_sq_out=None):
    """The float32 values of one tensor's 8-bit AdamW states, as a checkpoint
    stores them. Returns (exp_avg, exp_avg_sq)."""
    import torch
    what = "vcoll_adamw_unpack"
    n, dev = exp_avg.numel(), exp_avg.device
    groups = -(-n // ADAMW_GROUP)
    given = exp_avg_out is not None or exp_avg_sq_out is not None
    exp_avg_out = torch.empty(exp_avg.shape, device=dev) if exp_avg_out is None else exp_avg_out
    exp_avg_sq_out = torch.empty(exp_avg.shape, device=dev) if exp_avg_sq_out is None else exp_avg_sq_out
    ins, outs = (exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale), (exp_avg_out, exp_avg_sq_out)
    for t, kind, want in zip(ins + outs, (torch.uint8,) * 2 + (torch.float32,) * 4, (n, n, groups, groups, n, n)):
        if t.dtype is not kind or t.numel() != want or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{what}: expected a contiguous {kind} tensor of {want} elements on {dev}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    _on_current_gpu(exp_avg)
    if given:
        _no_overlap(list(ins), list(outs), what)
        _disjoint(list(outs), what)
    _check(_lib().vcoll_adamw_unpack(n, *[t.data_ptr() if n else None for t in ins + outs], _stream(exp_avg)), what)
    return exp_avg_out, exp_avg_sq_out
