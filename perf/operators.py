"""The training-step operators around the collectives, as work to measure.

Router (logits to chosen experts and weights, and its gradient), the sort of
(token, expert) pairs with the dispatch it steers, the weighted combine and
its gradient, and the AdamW step. ``own`` selects the framework's calls;
otherwise ``run`` evaluates the same formulas with elementary torch
operations in float32.

Rank buffers that differ in length (expert rows) are slices of one flat
[rows, hidden] tensor, rank 0's first.
"""
import math

import torch

own = False

GROUP = 128                                # elements per scale of an 8-bit optimiser state
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=100, grad_scale=0.125, seed=7)


def _vc():
    import collective_communication_algorithms_vcoll_amd as vc
    return vc


# -----------------------------------------------------------------------------
# cases


def _route(op, p, tokens, experts, topk, dtype, normalise, pad=0):
    return dict(op=op, p=p, tokens=tokens, experts=experts, topk=topk, dtype=dtype, normalise=normalise, pad=pad)


def _rows(op, p, tokens, experts, topk, hidden, dtype, weighted=True, pad=0):
    return dict(op=op, p=p, tokens=tokens, experts=experts, topk=topk, hidden=hidden, dtype=dtype, weighted=weighted,
                pad=pad)


def _adamw(count, total, param, grad, bits, align):
    return dict(op="adamw", count=count, total=total, param=param, grad=grad, bits=bits, align=align)


def listed():
    return [
        # one decoding step: one token on each of 8 ranks
        dict(_route("route", 8, 1, 256, 8, "f32", True), name="route decode 8x1 e256 k8 f32"),
        # the router of a training step of the 8 x 4096-token workload, a few padded tokens on every rank
        dict(_route("route", 8, 4096, 256, 8, "f32", True, 5), name="route train 8x4096 e256 k8 f32"),
        # its gradient where the weights are a softmax over all experts, logits kept in bf16
        dict(_route("route_bwd", 8, 4096, 256, 8, "bf16", False, 5), name="route grad 8x4096 e256 k8 bf16 all"),
        # a small layer of odd sizes, weights normalised over the chosen
        dict(_route("route_bwd", 5, 777, 60, 3, "f32", True), name="route grad 5x777 e60 k3 f32 norm"),
        # tokens to experts in a decoding step of 16 sequences a rank
        dict(_rows("sort", 8, 16, 256, 8, 7168, "bf16"), name="sort+dispatch decode 8x16 h7168 bf16"),
        # tokens to experts in a training step
        dict(_rows("sort", 8, 4096, 256, 8, 7168, "bf16", pad=5), name="sort+dispatch train 8x4096 h7168 bf16"),
        # experts' rows back to a training step's tokens, with the router's weights
        dict(_rows("combine", 8, 4096, 256, 8, 7168, "bf16", pad=5), name="combine train 8x4096 h7168 bf16"),
        # the dispatch's gradient (unit weights) on odd rows
        dict(_rows("combine", 4, 333, 24, 3, 1001, "f32", weighted=False), name="combine 4x333 h1001 f32 unit"),
        # the combine's gradient in a training step
        dict(_rows("combine_bwd", 8, 4096, 256, 8, 7168, "bf16", pad=5), name="combine grad 8x4096 h7168 bf16"),
        # and on the short batches of a fine-tuning step
        dict(_rows("combine_bwd", 8, 16, 256, 8, 7168, "bf16"), name="combine grad 8x16 h7168 bf16"),
        # the tensors of one 25 MiB gradient bucket, packed without gaps
        dict(_adamw(37, 6_553_600, "f32", "f32", 32, 1), name="adamw 37 tensors 25MiB f32 states32"),
        # the tensors behind 192 MiB of bf16 gradients, states in 8 bits
        dict(_adamw(150, 100_663_296, "bf16", "bf16", 8, 128), name="adamw 150 tensors 192MiB bf16 states8"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "sort", "combine", "combine_bwd", "adamw"])
    if op == "adamw":
        total = _log_int(rng, 1000, 60_000_000)
        param = rng.choice(["f32", "bf16"])
        bits = rng.choice([32, 8])
        return _adamw(min(_log_int(rng, 1, 200), total // 5), total, param, rng.choice(["f32", "bf16"]), bits,
                      128 if bits == 8 else rng.choice([1, 128]))
    p = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
    per_rank = _log_int(rng, 2, max(2, 512 // p))
    experts = p * per_rank
    topk = rng.randint(1, min(10, experts))
    tokens = _log_int(rng, 1, 32768 // p)
    dtype = rng.choice(["f32", "bf16"])
    pad = rng.choice([0, 0, rng.randint(0, tokens // 4)])
    if op in ("route", "route_bwd"):
        return _route(op, p, tokens, experts, topk, dtype, rng.random() < 0.5, pad)
    hidden = _log_int(rng, 16, 8192)
    if rng.random() < 0.7:
        hidden = max(8, hidden // 8 * 8)
    # no more rows than the listed training step has
    tokens = max(1, min(tokens, 400_000_000 // (p * topk * hidden)))
    return _rows(op, p, tokens, experts, topk, hidden, dtype, op != "combine" or rng.random() < 0.7,
                 min(pad, tokens // 4))


# -----------------------------------------------------------------------------
# inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _router_logits(case, g):
    """Popular experts have larger biases (Zipf 1.1, as the routing workload); padded tokens are masked whole."""
    p, t, e = case["p"], case["tokens"], case["experts"]
    bias = -1.1 * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
    z = torch.randn((p, t, e), device="cuda", generator=g) + bias
    if case["pad"]:
        z[:, t - case["pad"]:] = -math.inf
    return z.to(_dtype(case["dtype"]))


def _chosen(case, g):
    """Expert ids [p, tokens, topk] of Zipf popularity, distinct per token, -1 for padded tokens."""
    p, t, e = case["p"], case["tokens"], case["experts"]
    u = torch.rand((p, t, e), device="cuda", generator=g).clamp_(1e-7, 1 - 1e-7)
    z = -1.1 * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32)) - torch.log(-torch.log(u))
    ids = torch.topk(z, case["topk"], dim=-1).indices.to(torch.int32)
    if case["pad"]:
        ids[:, t - case["pad"]:] = -1
    return ids


def _tensor_sizes(count, total):
    """`count` tensor sizes of a model: small vectors next to matrices, their sum `total`."""
    raw = [4.0 ** (-(i % 5)) * (1 + 0.37 * ((i * 7) % 11)) for i in range(count)]
    left = total - count
    sizes = [1 + int(left * r / sum(raw)) for r in raw]
    sizes[0] += total - sum(sizes)
    return sizes


def _layout(case):
    """Start and size of every tensor in the flat buffer, and the buffer's length."""
    at, starts, sizes = 0, [], _tensor_sizes(case["count"], case["total"])
    for n in sizes:
        starts.append(at)
        at += -(-n // case["align"]) * case["align"]
    return starts, sizes, at


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "adamw":
        starts, sizes, total = _layout(case)
        s["starts"], s["sizes"] = starts, sizes
        live = torch.zeros(total, device="cuda", dtype=torch.bool)
        for a, n in zip(starts, sizes):
            live[a:a + n] = True
        s["grad"] = (torch.randn(total, device="cuda", generator=g) * 1e-3 * live).to(_dtype(case["grad"]))
        weights = torch.randn(total, device="cuda", generator=g) * 0.02 * live
        m = torch.randn(total, device="cuda", generator=g) * 1e-4 * live
        v = torch.randn(total, device="cuda", generator=g).square() * 1e-7 * live
        s["master"] = weights
        s["param"] = weights.to(torch.bfloat16) if case["param"] == "bf16" else weights
        if case["bits"] == 8:
            noise = _noise(s, total)
            s["m"], s["m_scale"] = _encode_m(m, noise)
            s["v"], s["v_scale"] = _encode_v(v, noise)
        else:
            s["m"], s["v"] = m, v
        if own:
            s["step"] = _own_adamw(s)
        return s
    if op in ("route", "route_bwd"):
        s["logits"] = _router_logits(case, g)
        if op == "route_bwd":
            s["ids"], s["weights"] = _plain_route(s["logits"], case["topk"], case["normalise"])
            s["d_weights"] = torch.randn(s["weights"].shape, device="cuda", generator=g)
        return s
    p, t, k, h, dt = case["p"], case["tokens"], case["topk"], case["hidden"], _dtype(case["dtype"])
    s["ids"] = _chosen(case, g)
    s["per_rank"] = case["experts"] // p
    slots, offsets = _plain_sort(s["ids"], s["per_rank"])
    s["rows"] = offsets[:, -1].tolist()
    total = sum(s["rows"])
    if op == "sort":
        s["tokens"] = torch.randn((p, t, h), device="cuda", generator=g).to(dt)
        s["recv"] = torch.empty((total, h), device="cuda", dtype=dt)
        s["recv_ranks"] = list(s["recv"].split(s["rows"]))
        return s
    s["expert_out"] = torch.empty((total, h), device="cuda", dtype=dt)
    s["expert_out"].normal_(generator=g)
    s["expert_ranks"] = list(s["expert_out"].split(s["rows"]))
    s["slots"] = slots
    s["weights"] = None
    if case["weighted"]:
        s["weights"] = torch.softmax(torch.randn((p, t, k), device="cuda", generator=g), dim=-1)
    if op == "combine_bwd":
        s["d_out"] = torch.randn((p, t, h), device="cuda", generator=g).to(dt)
        s["d_expert"] = torch.zeros((total, h), device="cuda", dtype=dt)
        s["d_expert_ranks"] = list(s["d_expert"].split(s["rows"]))
    return s


# -----------------------------------------------------------------------------
# plain forms


def _plain_route(logits, topk, normalise):
    z = logits.float()
    order, ids = torch.sort(z, dim=-1, descending=True, stable=True)
    top, ids = order[..., :topk], ids[..., :topk]
    live = top > -math.inf
    peak = top[..., :1].clamp(min=-3e38)
    e = torch.exp(top - peak)
    total = (e if normalise else torch.exp(z - peak)).sum(dim=-1, keepdim=True)
    weights = torch.where(live, e / total, torch.zeros_like(e))
    return torch.where(live, ids, torch.full_like(ids, -1)).to(torch.int32), weights


def _plain_route_backward(logits, ids, weights, d_weights, normalise):
    z = logits.float()
    live = ids >= 0
    at = ids.long().clamp(min=0)
    dw = torch.where(live, d_weights, torch.zeros_like(d_weights))
    mean = (weights * dw).sum(dim=-1, keepdim=True)
    if normalise:
        d = torch.zeros_like(z).scatter_add_(-1, at, weights * (dw - mean))
    else:
        peak = z.max(dim=-1, keepdim=True).values.clamp(min=-3e38)
        e = torch.exp(z - peak)
        total = e.sum(dim=-1, keepdim=True)
        prob = e / torch.where(total > 0, total, torch.ones_like(total))
        d = prob * (torch.zeros_like(z).scatter_add_(-1, at, dw) - mean)
    return d.to(logits.dtype)


def _plain_sort(ids, per_rank):
    """(slots [p, tokens*topk, 2], offsets [p, per_rank + 1]): the pairs in (rank, token, slot) order, stably by expert."""
    p = ids.shape[0]
    experts = p * per_rank
    key = ids.reshape(-1).long()
    key = torch.where((key >= 0) & (key < experts), key, torch.full_like(key, experts))
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.bincount(key, minlength=experts + 1)[:experts].reshape(p, per_rank)
    first = torch.cat([torch.zeros(1, dtype=torch.int64, device=key.device), counts.sum(dim=1).cumsum(0)])
    rank = key // per_rank
    gone = key == experts
    slots = torch.stack([torch.where(gone, -1, rank), torch.where(gone, -1, place - first[rank.clamp(max=p)])], dim=-1)
    offsets = torch.cat([torch.zeros((p, 1), dtype=torch.int64, device=key.device), counts.cumsum(dim=1)], dim=1)
    return slots.reshape(p, -1, 2).to(torch.int32), offsets.to(torch.int32)


def _flat_rows(slots, rows):
    """The row in the flat buffer of every pair, and which pairs have one."""
    first = torch.tensor([0] + rows[:-1], device=slots.device).cumsum(0)
    live = slots[..., 0] >= 0
    at = first[slots[..., 0].clamp(min=0).long()] + slots[..., 1]
    return torch.where(live, at, torch.zeros_like(at)), live


def _plain_dispatch(s, slots):
    p, t, h = s["tokens"].shape
    at, live = _flat_rows(slots, s["rows"])
    pair = torch.nonzero(live.reshape(-1)).reshape(-1)
    s["recv"][at.reshape(-1)[pair]] = s["tokens"].reshape(p * t, h)[pair // s["case"]["topk"]]
    return s["recv"]


def _gathered(s, dtype):
    """Every pair's expert row [p, tokens, topk, hidden]; zeros for a pair without one."""
    c = s["case"]
    shape = (c["p"], c["tokens"], c["topk"])
    at, live = _flat_rows(s["slots"], s["rows"])
    if s["expert_out"].shape[0] == 0:
        return torch.zeros((*shape, c["hidden"]), dtype=dtype, device="cuda"), at, live
    e = s["expert_out"][at.reshape(-1)].to(dtype).reshape(*shape, c["hidden"])
    return e.mul_(live.reshape(*shape, 1)), at, live


def _plain_combine(s):
    e, _, _ = _gathered(s, torch.float32)
    if s["weights"] is not None:
        e = e.mul_(s["weights"][..., None])
    return e.sum(dim=2).to(s["expert_out"].dtype)


def _plain_combine_backward(s):
    c = s["case"]
    e, at, live = _gathered(s, torch.float32)
    dy = s["d_out"].float()[:, :, None]
    d_weights = e.mul_(dy).sum(dim=-1)
    del e
    d = (s["weights"][..., None] * dy).to(s["expert_out"].dtype).reshape(-1, c["hidden"])
    pair = torch.nonzero(live.reshape(-1)).reshape(-1)
    s["d_expert"][at.reshape(-1)[pair]] = d[pair]
    return s["d_expert"], d_weights


# --- 8-bit optimiser states ---------------------------------------------------
# exp_avg is kept as E4M3 codes, exp_avg_sq as unsigned codes of 5 exponent and
# 3 fraction bits (value (8 + f) * 2^(e - 34), f * 2^-33 for e = 0), each with
# one power-of-two scale per 128 elements, rounded up or down at random: a
# 32-bit hash of the element gives the two 16-bit fractions to compare with.


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x85157AF5) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _noise(s, total):
    """The hash of every element of the flat buffer: of the seed, the step, the tensor's number and the element's."""
    starts = torch.tensor(s["starts"], device="cuda")
    ends = torch.cat([starts[1:], torch.tensor([total], device="cuda")])
    index = torch.arange(total, device="cuda") - starts.repeat_interleave(ends - starts)
    first = _mix((HYPER["seed"] + _mix(HYPER["step"])) & 0xFFFFFFFF)
    keys = [_mix((first + 0x9E3779B9 * k) & 0xFFFFFFFF) for k in range(len(s["starts"]))]
    key = torch.tensor(keys, device="cuda").repeat_interleave(ends - starts)
    return _mix(((index & 0xFFFFFFFF) + key + _mix(index >> 32)) & 0xFFFFFFFF)


def _bits(x):
    return x.view(torch.int32).long() & 0xFFFFFFFF


def _power(k):
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _grouped(x, fill=0.0):
    return torch.nn.functional.pad(x, (0, -x.numel() % GROUP), value=fill).reshape(-1, GROUP)


def _scale(x, fraction, above):
    """Per group the smallest power of two with max|x| <= top * scale, where `top` has this fraction and exponent."""
    u = _bits(_grouped(x.abs()).max(dim=1).values)
    k = (u >> 23) - above + ((u & 0x7FFFFF) > fraction)
    return torch.where(u == 0, torch.zeros_like(k), k.clamp(-126, 126))


def _encode_m(m, noise):
    k = _scale(m, 0x600000, 135)
    y = (_grouped(m) * _power(-k)[:, None]).reshape(-1)[:m.numel()]
    a = y.abs()
    r = (noise >> 16) << 4
    code = torch.where(a < 2.0 ** -6, ((a * 2.0 ** 29).long() + r) >> 20, ((_bits(a) + r) >> 20) - 960)
    return (code | torch.where(y < 0, 128, 0)).to(torch.uint8), _power(k)


def _encode_v(v, noise):
    k = _scale(v, 0x700000, 127)
    y = (_grouped(v) * _power(-k)[:, None]).reshape(-1)[:v.numel()]
    r = (noise & 0xFFFF) << 4
    code = torch.where(y < 2.0 ** -30, ((y * 2.0 ** 53).long() + r) >> 20, ((_bits(y) + r) >> 20) - 768)
    return code.to(torch.uint8), _power(k)


def _decode_m(code, scale):
    c = torch.arange(256, device="cuda")
    e, f = (c >> 3) & 15, c & 7
    value = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).double())) * torch.where(c < 128, 1.0, -1.0)
    return (_grouped(value.float()[code.int()]) * scale[:, None]).reshape(-1)[:code.numel()]


def _decode_v(code, scale):
    c = torch.arange(256, device="cuda")
    e, f = c >> 3, c & 7
    value = torch.where(e == 0, f * 2.0 ** -33, (8 + f) * torch.exp2((e - 34).double()))
    return (_grouped(value.float()[code.int()]) * scale[:, None]).reshape(-1)[:code.numel()]


def _plain_adamw(s):
    c, hy = s["case"], HYPER
    eight = c["bits"] == 8
    m = _decode_m(s["m"], s["m_scale"]) if eight else s["m"]
    v = _decode_v(s["v"], s["v_scale"]) if eight else s["v"]
    g = s["grad"].float() * hy["grad_scale"]
    m = m * hy["beta1"] + g * (1 - hy["beta1"])
    v = v * hy["beta2"] + (g * g) * (1 - hy["beta2"])
    bc1, bc2 = 1 - hy["beta1"] ** hy["step"], 1 - hy["beta2"] ** hy["step"]
    move = m / (torch.sqrt(v) * (1 / math.sqrt(bc2)) + hy["eps"])
    s["master"].copy_(s["master"] * (1 - hy["lr"] * hy["weight_decay"]) - move * (hy["lr"] / bc1))
    if c["param"] == "bf16":
        s["param"].copy_(s["master"])
    if eight:
        noise = _noise(s, m.numel())
        code, scale = _encode_m(m, noise)
        s["m"].copy_(code), s["m_scale"].copy_(scale)
        code, scale = _encode_v(v, noise)
        s["v"].copy_(code), s["v_scale"].copy_(scale)
        m, v = _decode_m(s["m"], s["m_scale"]), _decode_v(s["v"], s["v_scale"])
    else:
        m, v = s["m"].copy_(m), s["v"].copy_(v)
    return dict(param=s["param"], master=s["master"], exp_avg=m, exp_avg_sq=v)


# -----------------------------------------------------------------------------
# the framework's calls


def _slices(s, flat):
    return [flat[a:a + n] for a, n in zip(s["starts"], s["sizes"])]


def _scale_slices(s, flat):
    return [flat[a // GROUP:a // GROUP + -(-n // GROUP)] for a, n in zip(s["starts"], s["sizes"])]


def _own_adamw(s):
    """The optimiser that a training program keeps: it holds the tensors and their states."""
    eight = s["case"]["bits"] == 8
    return _vc().prepare_adamw(
        _slices(s, s["param"]), _slices(s, s["grad"]), _slices(s, s["m"]), _slices(s, s["v"]),
        master=_slices(s, s["master"]) if s["case"]["param"] == "bf16" else None,
        exp_avg_scale=_scale_slices(s, s["m_scale"]) if eight else None,
        exp_avg_sq_scale=_scale_slices(s, s["v_scale"]) if eight else None)


def _own_run(s):
    vc, c = _vc(), s["case"]
    op = c["op"]
    if op == "route":
        return vc.vcoll_moe_route(s["logits"], c["topk"], normalise=c["normalise"])
    if op == "route_bwd":
        return vc.vcoll_moe_route_backward(s["logits"], s["ids"], s["weights"], s["d_weights"], normalise=c["normalise"])
    if op == "sort":
        slots, offsets = vc.vcoll_moe_sort(s["ids"], s["per_rank"])
        vc.vcoll_moe_dispatch(list(s["tokens"]), list(slots), s["rows"], c["topk"], recv=s["recv_ranks"])
        return slots, offsets, s["recv"]
    if op == "combine":
        return vc.vcoll_moe_combine_weighted(s["expert_ranks"], s["slots"], s["weights"], c["tokens"], c["topk"])
    if op == "combine_bwd":
        _, d_weights = vc.vcoll_moe_combine_weighted_backward(s["d_out"], s["expert_ranks"], s["slots"], s["weights"],
                                                              c["topk"], d_expert_out=s["d_expert_ranks"])
        return s["d_expert"], d_weights
    s["step"](**HYPER)
    m, v = s["m"], s["v"]
    if c["bits"] == 8:                     # what the states stand for, as a checkpoint stores them
        m, v = vc.vcoll_adamw_unpack(m, v, s["m_scale"], s["v_scale"])
    return dict(param=s["param"], master=s["master"], exp_avg=m, exp_avg_sq=v)


def run(s):
    if own:
        return _own_run(s)
    c = s["case"]
    op = c["op"]
    if op == "route":
        return _plain_route(s["logits"], c["topk"], c["normalise"])
    if op == "route_bwd":
        return _plain_route_backward(s["logits"], s["ids"], s["weights"], s["d_weights"], c["normalise"])
    if op == "sort":
        slots, offsets = _plain_sort(s["ids"], s["per_rank"])
        return slots, offsets, _plain_dispatch(s, slots)
    if op == "combine":
        return _plain_combine(s)
    if op == "combine_bwd":
        return _plain_combine_backward(s)
    return _plain_adamw(s)


# -----------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "adamw":
        n = case["total"]
        grad = 2 if case["grad"] == "bf16" else 4
        state = 2 * 2 * (1 + 4 / GROUP) + 8 if case["bits"] == 8 else 2 * 8     # 8 bits: and the values they stand for
        return {"bytes": n * (8 + (2 if case["param"] == "bf16" else 0) + grad + state), "flops": 14.0 * n}
    es = 2 if case["dtype"] == "bf16" else 4
    tokens = case["p"] * case["tokens"]
    pairs = tokens * case["topk"]
    dense = tokens * case["experts"]
    if op == "route":
        return {"bytes": dense * es + pairs * 8, "flops": 2.0 * dense + 4.0 * pairs}
    if op == "route_bwd":
        return {"bytes": dense * es * (1 if case["normalise"] else 2) + pairs * 12, "flops": 4.0 * dense}
    live = case["p"] * (case["tokens"] - case["pad"])
    rows, h = live * case["topk"], case["hidden"]
    if op == "sort":
        return {"bytes": pairs * 12 + (case["experts"] + case["p"]) * 4 + (live + rows) * h * es, "flops": 0.0}
    weights = 4 * pairs if case["weighted"] else 0
    if op == "combine":
        return {"bytes": pairs * 8 + weights + (rows + tokens) * h * es, "flops": 2.0 * rows * h}
    return {"bytes": pairs * 12 + weights + (live + 2 * rows) * h * es, "flops": 3.0 * rows * h}


# -----------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_adamw(case, seed):
    s = prepare(dict(case), seed)
    hy = HYPER
    eight = case["bits"] == 8
    m = _decode_m(s["m"], s["m_scale"]).double() if eight else s["m"].double()
    v = _decode_v(s["v"], s["v_scale"]).double() if eight else s["v"].double()
    g = s["grad"].double() * hy["grad_scale"]
    m = hy["beta1"] * m + (1 - hy["beta1"]) * g
    v = hy["beta2"] * v + (1 - hy["beta2"]) * g * g
    m_hat, v_hat = m / (1 - hy["beta1"] ** hy["step"]), v / (1 - hy["beta2"] ** hy["step"])
    w = s["master"].double()
    w = w - hy["lr"] * hy["weight_decay"] * w - hy["lr"] * m_hat / (torch.sqrt(v_hat) + hy["eps"])
    if eight:                              # one of two neighbouring codes: at a border of the choice no value is exact
        m = v = None
    return dict(param=w, master=w, exp_avg=m, exp_avg_sq=v)


def exact(case, seed):
    global own
    kept, own = own, False                 # the inputs alone, without the framework's objects
    try:
        op = case["op"]
        if op == "adamw":
            return _exact_adamw(case, seed)
        s = prepare(dict(case), seed)
    finally:
        own = kept
    if op == "route":
        z = s["logits"].double()
        top = torch.sort(z, dim=-1, descending=True).values[..., :case["topk"]]
        among = top if case["normalise"] else z
        return None, torch.nan_to_num(torch.exp(top - torch.logsumexp(among, dim=-1, keepdim=True)), nan=0.0)
    if op == "route_bwd":
        z = s["logits"].double()
        at = s["ids"].long()
        chosen = torch.zeros(z.shape, dtype=torch.float64, device="cuda")
        chosen.scatter_(-1, at.clamp(min=0), (at >= 0).double())
        masked = torch.where(chosen > 0, z, torch.full_like(z, -math.inf)) if case["normalise"] else z
        prob = torch.nan_to_num(torch.softmax(masked, dim=-1), nan=0.0)
        dw = torch.zeros_like(z).scatter_(-1, at.clamp(min=0), s["d_weights"].double() * (at >= 0))
        return prob * (dw - (prob * dw).sum(dim=-1, keepdim=True))
    if op == "sort":
        return None
    e, at, live = _gathered(s, torch.float64)
    if op == "combine":
        if s["weights"] is not None:
            e = e.mul_(s["weights"].double()[..., None])
        return e.sum(dim=2)
    dy = s["d_out"].double()
    d_weights = torch.stack([(e[:, :, k] * dy).sum(dim=-1) for k in range(case["topk"])], dim=-1)
    del e
    d = torch.zeros(s["d_expert"].shape, dtype=torch.float64, device="cuda")
    for k in range(case["topk"]):
        keep = live.reshape(*s["weights"].shape)[..., k]
        d[at.reshape(*s["weights"].shape)[..., k][keep]] = (s["weights"][..., k, None].double() * dy)[keep]
    return d, d_weights
