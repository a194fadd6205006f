"""Training-step operators on the CPU: the oracle against hand cases,
differences and independent formulas, and every refusal of the C entry points
and of the binding (nothing is launched)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import collective_communication_algorithms_vcoll_amd as vc
from oracle import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "collective_communication_algorithms_vcoll_amd", "csrc")
ROCM_INCLUDE = "/opt/rocm/include"


# --- the oracle -----------------------------------------------------------------

def test_route_by_hand():
    z = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, -0.0, -1.0, 2.0]])
    ids, w = train.route(z, 3, True)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [3, 0, 1]]
    e = np.exp(-2.0)
    assert np.allclose(w[0], [1 / (2 + e), 1 / (2 + e), e / (2 + e)], rtol=1e-15)
    assert w[1].tolist() == [0, 0, 0]
    _, w_all = train.route(z, 1, False)
    assert np.isclose(w_all[2, 0], np.exp(2.0) / (np.exp(2.0) + 2 + np.exp(-1.0)), rtol=1e-15)


@pytest.mark.parametrize("normalise", [True, False])
def test_route_gradient_against_differences(normalise):
    rng = np.random.default_rng(3)
    z = rng.normal(size=(4, 7)) * 2
    z[1, 2] = z[2, :] = -np.inf
    ids, _ = train.route(z, 3, normalise)
    dw = rng.normal(size=(4, 3))
    dz = train.route_backward(z, ids, dw, normalise)
    h = 1e-6
    for t in range(4):
        for e in range(7):
            if not np.isfinite(z[t, e]):
                assert dz[t, e] == 0
                continue
            zp, zm = z.copy(), z.copy()
            zp[t, e] += h
            zm[t, e] -= h
            num = ((train.route(zp, 3, normalise)[1] - train.route(zm, 3, normalise)[1]) * dw).sum() / (2 * h)
            # second-order error of central differences: h^2 times a third derivative of size <= 10
            assert abs(num - dz[t, e]) < 1e-9 + 10 * h * h + 4 * 2.0 ** -52 / h


def test_sort_by_hand():
    # 2 ranks, 2 tokens, top-2 of 4 experts (2 per rank); rank 1's token 0 is masked in its second slot
    ids = np.array([[[3, 0], [1, 0]], [[0, -1], [2, 3]]], np.int32)
    slots, offsets = train.expert_sort(ids, 2)
    assert offsets.tolist() == [[0, 3, 4], [0, 1, 3]]
    assert slots.tolist() == [[[1, 1], [0, 0], [0, 3], [0, 1]], [[0, 2], [-1, -1], [1, 0], [1, 2]]]


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(4)
    ids = np.array([[[1, 0], [2, -1]]], np.int32)
    slots, _ = train.expert_sort(ids, 3)
    e = [rng.normal(size=(3, 5))]
    w = rng.normal(size=(1, 2, 2))
    dy = rng.normal(size=(1, 2, 5))
    de, dw, _ = train.combine_weighted_backward(dy, e, slots, w, 2)
    f = lambda e, w: (train.combine_weighted(e, slots, w, 2, 2)[0] * dy).sum()          # noqa: E731
    h = 1e-6
    for x, d in ((w, dw), (e[0], de[0])):
        for at in np.ndindex(x.shape):
            was = x[at]
            x[at] = was + h
            up = f(e, w)
            x[at] = was - h
            num = (up - f(e, w)) / (2 * h)
            x[at] = was
            # linear in each argument: rounding of f (|f| < 100) over 2 h
            assert abs(num - d[at]) < 100 * 2.0 ** -52 / h


def test_m_codes_are_e4m3():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    got = train.decode_m(codes, np.ones(2, np.float32))
    assert np.array_equal(np.nan_to_num(got, nan=-1e9), np.nan_to_num(want, nan=-1e9))


def test_rounding_keeps_representable_values():
    """A value that a code stands for is kept whatever the random bits."""
    for fmt in (train.M_FORMAT, train.V_FORMAT):
        codes = np.arange(0x7F if fmt is train.M_FORMAT else 0x100)
        for up in (0, 0xFFFF << 4):
            assert np.array_equal(fmt.round(fmt.value(codes), np.full(codes.size, up)), codes)


def test_rounding_is_unbiased_and_to_a_neighbour():
    """The mean over the element hash is the value, within 6 standard errors."""
    n = 1 << 16
    bits = train.rounding_bits(n, 7, 3, 1)
    rng = np.random.default_rng(5)
    for fmt, up in ((train.M_FORMAT, (bits >> np.uint64(16)) << np.uint64(4)),
                    (train.V_FORMAT, (bits & np.uint64(0xFFFF)) << np.uint64(4))):
        for y in rng.uniform(0, fmt.top, 8).astype(np.float32).tolist() + [fmt.top * 2.0 ** -16, 2.0 ** (fmt.low - 4)]:
            got = fmt.value(fmt.round(np.full(n, y), up))
            lo, hi = np.unique(got)[[0, -1]]
            assert lo <= y <= hi and np.unique(got).size <= 2
            # 16 random bits: the probability of rounding up is off by less than 2^-16
            assert abs(got.mean() - y) <= 6 * (hi - lo) / 2 / np.sqrt(n) + (hi - lo) * 2.0 ** -16


def test_random_bits_have_no_visible_structure():
    """Means of the two halves, neighbours, steps, seeds and tensors are uncorrelated (5 standard errors)."""
    n = 1 << 16
    base = train.rounding_bits(n, 7, 3, 1)
    unit = lambda b: (b.astype(np.float64) + 0.5) / 65536 - 0.5                              # noqa: E731
    hi, lo = unit(base >> np.uint64(16)), unit(base & np.uint64(0xFFFF))
    tol = 5 / np.sqrt(n)
    assert abs(hi.mean()) < tol and abs(lo.mean()) < tol
    others = [np.roll(hi, 1), lo] + [unit(train.rounding_bits(n, *k) >> np.uint64(16))
                                     for k in ((8, 3, 1), (7, 4, 1), (7, 3, 2), (7, 2, 1))]
    for x in others:
        assert abs(12 * (hi * x).mean()) < tol


def test_adamw_by_hand():
    """First step from zero states: m_hat = g, v_hat = g^2, so x moves by lr * sign(g) after its decay."""
    x = np.array([1.0, -2.0, 0.5], np.float32)
    g = np.array([0.25, -4.0, 0.0], np.float32)
    z = np.zeros(3, np.float32)
    y, m, v = train.adamw(x, g, z, z, lr=0.1, beta1=0.9, beta2=0.999, eps=1e-12, weight_decay=0.5, step=1, grad_scale=1)
    # ten float32 roundings of quantities of the size of x
    assert np.allclose(y, x * 0.95 - 0.1 * np.sign(g), rtol=10 * 2.0 ** -24, atol=0)
    assert np.allclose(m, 0.1 * g, rtol=2.0 ** -22) and np.allclose(v, 0.001 * g * g, rtol=2.0 ** -22)


def test_eight_bit_second_moment_decays():
    """Without gradients v shrinks by beta2 a step; rounding to nearest would leave it where it is."""
    v = np.full(4096, 1e-4, np.float32)
    code, s = train.encode_v(v, train.rounding_bits(4096, 1, 0, 0))
    for step in range(1, 501):
        _, _, v = train.adamw(v, np.zeros_like(v), np.zeros_like(v), train.decode_v(code, s), lr=0, beta1=0.9,
                              beta2=0.999, eps=1e-8, weight_decay=0, step=step, grad_scale=1)
        code, s = train.encode_v(v, train.rounding_bits(4096, 1, step, 0))
    want = 1e-4 * 0.999 ** 500
    # a code step is at most 1/8 of the value and is taken with probability <= 0.016 a step: after 500 steps the
    # value of one element varies by less than 1/8 * sqrt(500 * 0.016) < 0.36 of it; the mean of 4096 by 1/64 of that
    assert abs(train.decode_v(code, s).mean() / want - 1) < 6 * 0.36 / 64


# --- refusals of the C entry points ----------------------------------------------

ADDR = 1 << 20                    # an address for calls that are refused before it is used
INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3


def table(*addresses):
    return (ctypes.c_void_p * len(addresses))(*addresses)


def rows(*n):
    return (ctypes.c_int64 * len(n))(*n)


def call_route(p=1, tokens=4, experts=8, topk=2, dtype=0, logits=(ADDR,), ids=(ADDR,), weights=(ADDR,)):
    return vc._lib().vcoll_moe_route(p, tokens, experts, topk, dtype, 1, table(*logits), table(*ids), table(*weights),
                                     None)


@pytest.mark.parametrize("change,status", [
    (dict(p=0), INVALID), (dict(p=129), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=2 ** 48 + 1), INVALID),
    (dict(experts=0), INVALID), (dict(topk=0), INVALID), (dict(topk=9), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=7), INVALID), (dict(tokens=2 ** 31), INVALID), (dict(experts=1025), UNSUPPORTED),
    (dict(experts=100, topk=65), UNSUPPORTED), (dict(tokens=2 ** 27), UNSUPPORTED), (dict(logits=(None,)), INVALID),
    (dict(ids=(None,)), INVALID), (dict(weights=(None,)), INVALID), (dict(logits=(ADDR + 2,)), INVALID),
    (dict(dtype=1, logits=(ADDR + 1,)), INVALID), (dict(ids=(ADDR + 2,)), INVALID), (dict(weights=(ADDR + 1,)), INVALID),
])
def test_route_refusals(change, status):
    assert call_route(**change) == status


def test_nothing_to_route_is_fine():
    assert call_route(tokens=0, logits=(None,), ids=(None,), weights=(None,)) == 0


def call_route_backward(p=1, tokens=4, experts=8, topk=2, dtype=0, normalise=1, logits=(ADDR,), ids=(ADDR,),
                        weights=(ADDR,), d_weights=(ADDR,), d_logits=(ADDR,)):
    return vc._lib().vcoll_moe_route_backward(p, tokens, experts, topk, dtype, normalise, table(*logits), table(*ids),
                                              table(*weights), table(*d_weights), table(*d_logits), None)


@pytest.mark.parametrize("change,status", [
    (dict(p=0), INVALID), (dict(tokens=-1), INVALID), (dict(experts=0), INVALID), (dict(topk=9), INVALID),
    (dict(dtype=2), INVALID), (dict(experts=1025), UNSUPPORTED), (dict(normalise=0, logits=(None,)), INVALID),
    (dict(ids=(None,)), INVALID), (dict(weights=(None,)), INVALID), (dict(d_weights=(None,)), INVALID),
    (dict(d_logits=(None,)), INVALID), (dict(normalise=0, logits=(ADDR + 2,)), INVALID),
    (dict(d_logits=(ADDR + 2,)), INVALID), (dict(d_weights=(ADDR + 2,)), INVALID),
])
def test_route_backward_refusals(change, status):
    assert call_route_backward(**change) == status


def call_sort(p=1, tokens=4, topk=2, per_rank=8, ids=(ADDR,), slots=(ADDR,), offsets=ADDR, workspace=None, size=0):
    return vc._lib().vcoll_moe_sort(p, tokens, topk, per_rank, table(*ids), table(*slots), offsets, workspace, size, None)


@pytest.mark.parametrize("change,status", [
    (dict(p=0), INVALID), (dict(p=129), INVALID), (dict(tokens=-1), INVALID), (dict(topk=0), INVALID),
    (dict(per_rank=0), INVALID), (dict(tokens=2 ** 31), INVALID), (dict(p=2, tokens=2 ** 30, topk=1), INVALID),
    (dict(per_rank=1025), UNSUPPORTED), (dict(p=128, per_rank=9), UNSUPPORTED), (dict(ids=(None,)), INVALID),
    (dict(slots=(None,)), INVALID), (dict(offsets=None), INVALID), (dict(slots=(ADDR + 4,)), INVALID),
    (dict(ids=(ADDR + 2,)), INVALID), (dict(offsets=ADDR + 2), INVALID),
    (dict(tokens=5000), TOO_SMALL), (dict(tokens=5000, workspace=ADDR, size=10), TOO_SMALL),
    (dict(tokens=5000, workspace=None, size=1 << 20), INVALID), (dict(tokens=5000, workspace=ADDR + 1, size=1 << 20),
                                                                 INVALID),
])
def test_sort_refusals(change, status):
    assert call_sort(**change) == status


def test_sort_workspace():
    assert vc.vcoll_moe_sort_workspace(8, 16, 8, 32) == 0
    assert vc.vcoll_moe_sort_workspace(1, 0, 1, 1) == 0
    big = vc.vcoll_moe_sort_workspace(8, 4096, 8, 32)
    assert 0 < big <= 1 << 20
    assert vc.vcoll_moe_sort_workspace(1, 2 ** 31 - 1, 1, 1024) <= 1 << 20
    with pytest.raises(vc.VcollError):
        vc.vcoll_moe_sort_workspace(8, -1, 8, 32)


def call_combine(p=1, tokens=4, topk=2, hidden=16, dtype=0, e=(ADDR,), n=(8,), slots=(ADDR,), weights=(ADDR,),
                 out=(ADDR,)):
    return vc._lib().vcoll_moe_combine_weighted(p, tokens, topk, hidden, dtype, table(*e), rows(*n), table(*slots),
                                                table(*weights) if weights else None, table(*out), None)


@pytest.mark.parametrize("change,status", [
    (dict(p=0), INVALID), (dict(tokens=-1), INVALID), (dict(topk=0), INVALID), (dict(hidden=-1), INVALID),
    (dict(hidden=2 ** 31), INVALID), (dict(dtype=2), INVALID), (dict(n=(-1,)), INVALID), (dict(n=(2 ** 31,)), INVALID),
    (dict(tokens=2 ** 30), INVALID), (dict(tokens=2 ** 27), UNSUPPORTED), (dict(e=(None,)), INVALID),
    (dict(slots=(None,)), INVALID), (dict(weights=(None,)), INVALID), (dict(out=(None,)), INVALID),
    (dict(e=(ADDR + 2,)), INVALID), (dict(out=(ADDR + 1,), dtype=1), INVALID), (dict(weights=(ADDR + 2,)), INVALID),
    (dict(slots=(ADDR + 2,)), INVALID),
])
def test_combine_refusals(change, status):
    assert call_combine(**change) == status


def test_nothing_to_combine_is_fine():
    assert call_combine(tokens=0) == 0 and call_combine(hidden=0) == 0


def call_combine_backward(p=1, tokens=4, topk=2, hidden=16, dtype=0, dy=(ADDR,), e=(ADDR,), n=(8,), slots=(ADDR,),
                          weights=(ADDR,), de=(ADDR,), dw=(ADDR,)):
    return vc._lib().vcoll_moe_combine_weighted_backward(p, tokens, topk, hidden, dtype, table(*dy), table(*e), rows(*n),
                                                         table(*slots), table(*weights), table(*de), table(*dw), None)


@pytest.mark.parametrize("change,status", [
    (dict(p=0), INVALID), (dict(tokens=-1), INVALID), (dict(topk=0), INVALID), (dict(hidden=0), INVALID),
    (dict(dtype=2), INVALID), (dict(n=(-1,)), INVALID), (dict(tokens=2 ** 27), UNSUPPORTED), (dict(dy=(None,)), INVALID),
    (dict(e=(None,)), INVALID), (dict(slots=(None,)), INVALID), (dict(weights=(None,)), INVALID),
    (dict(de=(None,)), INVALID), (dict(dw=(None,)), INVALID), (dict(dy=(ADDR + 2,)), INVALID),
    (dict(e=(ADDR + 2,)), INVALID), (dict(de=(ADDR + 2,)), INVALID), (dict(dw=(ADDR + 2,)), INVALID),
])
def test_combine_backward_refusals(change, status):
    assert call_combine_backward(**change) == status


def call_adamw(count=1, param=0, grad=0, bits=32, hyper=None, null_hyper=False, null_tensors=False, **fields):
    from collective_communication_algorithms_vcoll_amd.training import _AdamwHyper, _AdamwTensor
    h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0, step=1, seed=0)
    h.update(hyper or {})
    t = dict(n=8, param=ADDR, grad=ADDR, master=ADDR, exp_avg=ADDR, exp_avg_sq=ADDR, exp_avg_scale=ADDR,
             exp_avg_sq_scale=ADDR)
    t.update(fields)
    tensors, hy = (_AdamwTensor * 1)(_AdamwTensor(**t)), _AdamwHyper(**h)
    return vc._lib().vcoll_adamw(count, None if null_tensors else tensors, param, grad, bits,
                                 None if null_hyper else ctypes.byref(hy), None)


@pytest.mark.parametrize("change,status", [
    (dict(count=-1), INVALID), (dict(param=2), INVALID), (dict(grad=2), INVALID), (dict(bits=16), INVALID),
    (dict(null_hyper=True), INVALID), (dict(null_tensors=True), INVALID), (dict(n=-1), INVALID),
    (dict(n=2 ** 48), UNSUPPORTED), (dict(param=0, exp_avg=None), INVALID), (dict(exp_avg_sq=None), INVALID),
    (dict(grad=1, bits=8, exp_avg_scale=None), INVALID), (dict(bits=8, exp_avg_sq_scale=ADDR + 2), INVALID),
    (dict(param=1, master=None), INVALID), (dict(param=1, master=ADDR + 2), INVALID), (dict(exp_avg=ADDR + 2), INVALID),
    *[(dict(hyper=h), INVALID) for h in (
        dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1),
        dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1e-8), dict(weight_decay=-1.0), dict(step=0),
        dict(grad_scale=float("inf")))],
])
def test_adamw_refusals(change, status):
    assert call_adamw(**change) == status


def test_nothing_to_update_is_fine():
    assert call_adamw(count=0) == 0 and call_adamw(n=0) == 0


def test_unpack_refusals():
    f = vc._lib().vcoll_adamw_unpack
    assert f(0, *[None] * 6, None) == 0
    assert f(-1, *[ADDR] * 6, None) == INVALID
    assert f(2 ** 48, *[ADDR] * 6, None) == UNSUPPORTED
    for k in range(6):
        a = [ADDR] * 6
        a[k] = None
        assert f(8, *a, None) == INVALID
        if k >= 2:
            a[k] = ADDR + 2
            assert f(8, *a, None) == INVALID


# --- refusals of the binding ------------------------------------------------------

def test_binding_refuses_wrong_buffers():
    import torch
    z = torch.zeros((2, 4, 8))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)                                         # noqa: E731
    f32 = torch.zeros
    bad = [
        lambda: vc.vcoll_moe_route(z, 0), lambda: vc.vcoll_moe_route(z, 9), lambda: vc.vcoll_moe_route(z[0], 2),
        lambda: vc.vcoll_moe_route([], 2), lambda: vc.vcoll_moe_route(z.transpose(1, 2), 2),
        lambda: vc.vcoll_moe_route([z[0], z[1, :3]], 2), lambda: vc.vcoll_moe_route(z, 2),
        lambda: vc.vcoll_moe_route_backward(z, i32(2, 4, 9), f32(2, 4, 9), f32(2, 4, 9)),
        lambda: vc.vcoll_moe_route_backward(z, i32(2, 4, 2), f32(2, 4, 3), f32(2, 4, 2)),
        lambda: vc.vcoll_moe_route_backward(z, f32(2, 4, 2), f32(2, 4, 2), f32(2, 4, 2)),
        lambda: vc.vcoll_moe_route_backward(z, i32(2, 4, 2), f32(2, 4, 2), f32(2, 4, 2)),
        lambda: vc.vcoll_moe_sort(f32(2, 4, 2), 4), lambda: vc.vcoll_moe_sort(i32(2, 4, 2), 0),
        lambda: vc.vcoll_moe_sort(i32(2, 4), 4), lambda: vc.vcoll_moe_sort(i32(2, 4, 2), 4),
        lambda: vc.vcoll_moe_combine_weighted([f32(3, 8)], i32(2, 8, 2), None, 4, 2),
        lambda: vc.vcoll_moe_combine_weighted([f32(3, 8)] * 2, i32(2, 8, 2), f32(2, 4, 3), 4, 2),
        lambda: vc.vcoll_moe_combine_weighted([f32(3, 8)] * 2, i32(2, 7, 2), None, 4, 2),
        lambda: vc.vcoll_moe_combine_weighted([f32(3, 8)] * 2, i32(2, 8, 2), None, 4, 2),
        lambda: vc.vcoll_moe_combine_weighted_backward(f32(2, 4, 8), [f32(3, 7)] * 2, i32(2, 8, 2), f32(2, 4, 2), 2),
        lambda: vc.vcoll_moe_combine_weighted_backward(f32(2, 4, 8), [f32(3, 8)] * 2, i32(2, 8, 2), f32(2, 4, 2), 2),
        lambda: vc.vcoll_adamw([f32(4)], [f32(5)], [f32(4)], [f32(4)], lr=1.0, step=1),
        lambda: vc.vcoll_adamw([f32(4)], [f32(4)], [f32(4)], [], lr=1.0, step=1),
        lambda: vc.vcoll_adamw([f32(4).bfloat16()], [f32(4)], [f32(4)], [f32(4)], lr=1.0, step=1),
        lambda: vc.vcoll_adamw([f32(4)], [f32(4)], [f32(4)], [f32(4)], master=[f32(4)], lr=1.0, step=1),
        lambda: vc.vcoll_adamw([f32(4)], [f32(4)], [f32(4)], [f32(4)], exp_avg_scale=[f32(1)], lr=1.0, step=1),
        lambda: vc.vcoll_adamw([f32(4)], [f32(4)], [f32(4)], [f32(4)], lr=1.0, step=1),
        lambda: vc.vcoll_adamw_unpack(*[torch.zeros(4, dtype=torch.uint8)] * 2, f32(1), f32(2)),
        lambda: vc.vcoll_adamw_unpack(*[torch.zeros(4, dtype=torch.uint8)] * 2, f32(1), f32(1)),
        lambda: vc.adamw_state([f32(4)], bits=16),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {k} was accepted")
    for f in (lambda: vc.vcoll_moe_route(z.double(), 2),
              lambda: vc.vcoll_adamw([f32(4).double()], [f32(4)], [f32(4)], [f32(4)], lr=1.0, step=1),
              lambda: vc.vcoll_adamw([f32(4)], [f32(4)], [f32(4).half()], [f32(4)], lr=1.0, step=1)):
        with pytest.raises(TypeError):
            f()


def test_overlap_sweep_agrees_with_pairwise_comparison():
    import torch
    flat = torch.zeros(64, dtype=torch.uint8)
    rng = np.random.default_rng(1)
    seen = set()
    for _ in range(4000):
        span = lambda: (lambda a, n: flat[a:a + n])(*(int(x) for x in rng.integers(0, (56, 9))))   # noqa: E731
        ins, outs = [span() for _ in range(rng.integers(0, 4))], [span() for _ in range(rng.integers(0, 4))]
        meet = lambda x, y: x.numel() and y.numel() and x.data_ptr() < y.data_ptr() + y.numel() \
            and y.data_ptr() < x.data_ptr() + x.numel()                                           # noqa: E731
        want = any(meet(x, y) for k, x in enumerate(outs) for y in outs[k + 1:] + ins)
        try:
            vc._apart(ins, outs, "test")
            got = False
        except ValueError:
            got = True
        assert got == bool(want)
        seen.add(got)
    assert seen == {True, False}


def test_binding_steps_over_no_tensors():
    vc.vcoll_adamw([], [], [], [], lr=1e-3, step=1)


# --- host half under sanitizers -----------------------------------------------------

@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE), reason="no g++ or HIP headers")
def test_entry_points_are_clean_under_asan_and_ubsan(tmp_path):
    exe = str(tmp_path / "train_sanitize")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", f"-I{ROCM_INCLUDE}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           os.path.join(ROOT, "tests", "c", "train_sanitize.cpp"), os.path.join(CSRC, "train_api.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert res.returncode == 0 and res.stdout.startswith("OK"), (res.stdout + res.stderr)[-4000:]
