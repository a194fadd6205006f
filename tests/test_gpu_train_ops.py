"""Training-step operators on the GPU against their definitions in 64 bits
(AdamW: against its float32 definition, bit for bit).

Tolerances count roundings, each off by at most half a step: u = 2^-24 of
float32, half_step(t) of a stored type.
"""
import numpy as np
import pytest

from oracle import train
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def vc():
    import torch
    assert torch.cuda.is_available()
    import collective_communication_algorithms_vcoll_amd as m
    return m


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def half_step(name):
    return {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[name]


def put(x, name="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt(name))


def get(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol) & ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} want {want[bad][0]} +- {np.broadcast_to(tol, got.shape)[bad][0]}"


# --- router -----------------------------------------------------------------------

def logits(p, T, E, name, seed, mask):
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(p, T, E)) * 3
    if mask:
        z[rng.random((p, T, E)) < 0.3] = -np.inf
        z[:, ::3] = -np.inf                                  # tokens masked whole
        if T > 1:
            z[:, 1, 1:] = -np.inf                            # one expert left
    z = put(z, name)
    return z, get(z)


ROUTES = [(1, 1, 1, 1, "f32", False), (1, 1, 256, 8, "f32", False), (2, 5, 7, 7, "bf16", True),
          (3, 17, 64, 64, "f32", True), (5, 9, 65, 3, "bf16", True), (2, 33, 128, 2, "f32", True),
          (8, 6, 256, 8, "bf16", False), (1, 40, 255, 10, "f32", True), (2, 11, 300, 8, "f32", True),
          (1, 7, 512, 6, "bf16", False), (1, 9, 1024, 8, "f32", True), (1, 5, 1000, 64, "bf16", True),
          (2, 9, 480, 7, "bf16", True), (1, 7, 770, 8, "f32", True),
          (1, 6, 100, 33, "f32", True), (1, 6, 250, 17, "bf16", False), (1, 5, 600, 40, "f32", True),
          (40, 2, 24, 2, "f32", True), (128, 1, 16, 1, "bf16", False), (1, 1, 130, 5, "f32", False)]


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("p,T,E,K,name,mask", ROUTES)
def test_route(vc, p, T, E, K, name, mask, normalise):
    z, z64 = logits(p, T, E, name, E * 7 + K, mask)
    ids, w = vc.vcoll_moe_route(z, K, normalise=normalise)
    for i in range(p):
        want_ids, want = train.route(z64[i], K, normalise)
        assert np.array_equal(get(ids[i]), want_ids), f"rank {i}"
        # exp's argument is off by u times its size (< 50) and exp by 2 u; E such terms are added in float32 along a
        # chain of at most 16 + 6 additions, and there is one division
        close(get(w[i]), want, (2 * 50 + 40) * U * want + 2.0 ** -126, f"rank {i} weights")


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("p,T,E,K,name,mask", ROUTES)
def test_route_backward(vc, p, T, E, K, name, mask, normalise):
    z, z64 = logits(p, T, E, name, E * 5 + K, mask)
    ids, w = vc.vcoll_moe_route(z, K, normalise=normalise)
    dw = put(np.random.default_rng(E).normal(size=(p, T, K)))
    dz = vc.vcoll_moe_route_backward(z, ids, w, dw, normalise=normalise)
    for i in range(p):
        want = train.route_backward(z64[i], get(ids[i]), get(dw[i]), normalise)
        # q and w are as far off as above; the mean adds K products along a chain of 6, then a difference and a product
        size = np.abs(get(dw[i])).max(axis=1, initial=0)[:, None]
        _, q = train.route(z64[i], E, normalise=False)
        q = np.ones_like(want) if normalise else np.where(z64[i] > -np.inf, 1.0, 0.0)
        close(get(dz[i]), want, (2 * (2 * 50 + 40) + 16) * U * 2 * size * q + half_step(name) * np.abs(want) + 2.0 ** -126,
              f"rank {i}")


def test_route_gradient_against_differences(vc):
    """Differences of the GPU's own forward pass."""
    z, z64 = logits(1, 6, 12, "f32", 3, True)
    rng = np.random.default_rng(4)
    dw = rng.normal(size=(1, 6, 4))
    for normalise in (True, False):
        ids, w = vc.vcoll_moe_route(z, 4, normalise=normalise)
        got = get(vc.vcoll_moe_route_backward(z, ids, w, put(dw), normalise=normalise))
        h = 2.0 ** -7                                        # exact next to logits of size < 16
        for e in range(12):
            step = np.zeros(z64.shape)
            step[..., e] = h
            up, dn = (vc.vcoll_moe_route(put(z64 + s * step), 4, normalise=normalise) for s in (1, -1))
            same = (get(up[0]) == get(ids)).all(axis=-1) & (get(dn[0]) == get(ids)).all(axis=-1)
            num = ((get(up[1]) - get(dn[1])) * dw).sum(axis=-1) / (2 * h)
            # h^2/6 times third derivatives (< 1 per weight), and two forward errors over 2 h
            tol = (h * h + 2 * (2 * 50 + 40) * U / (2 * h)) * np.abs(dw).sum(axis=-1)
            assert (np.abs(num - got[..., e]) <= tol)[same].all(), e
            assert same.sum() >= 4


def test_route_ties_and_zeros(vc):
    z = np.zeros((1, 3, 200))
    z[0, 0] = np.where(np.arange(200) % 2, 0.0, -0.0)        # all equal
    z[0, 1, 150] = z[0, 1, 37] = 1.0
    z[0, 2, :] = -5.0
    for name in ("f32", "bf16"):
        ids, _ = vc.vcoll_moe_route(put(z, name), 5)
        assert get(ids[0]).tolist() == [[0, 1, 2, 3, 4], [37, 150, 0, 1, 2], [0, 1, 2, 3, 4]]


def test_route_values_at_the_edges(vc):
    """NaN, infinities, the type's lowest and largest values, denormals."""
    big = 3.4028234663852886e38
    z = np.full((1, 6, 70), -1.0)
    z[0, 0, 66] = np.nan
    z[0, 1, 5] = np.inf
    z[0, 2, :] = -big
    z[0, 3, :] = -big
    z[0, 3, 69] = big
    z[0, 4, :] = -np.inf
    z[0, 4, 68] = -big
    z[0, 5, 64], z[0, 5, 3] = 2.0 ** -149, 2.0 ** -148
    for normalise in (True, False):
        ids, w = vc.vcoll_moe_route(put(z), 2, normalise=normalise)
        want_ids, want = train.route(z[0], 2, normalise)
        assert np.array_equal(get(ids[0]), want_ids)
        close(get(w[0]), want, 64 * U * np.abs(np.nan_to_num(want)), "weights")
        dz = get(vc.vcoll_moe_route_backward(put(z), ids, w, put(np.ones((1, 6, 2))), normalise=normalise))
        assert np.isfinite(dz[0, 2:]).all() and (dz[0, 4, :68] == 0).all()


def shifted(x, by=1):
    """A copy of x that starts `by` elements off its allocation's alignment."""
    import torch
    flat = torch.empty(x.numel() + by, dtype=x.dtype, device="cuda")
    y = flat[by:].view(x.shape)
    y.copy_(x)
    return y


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_route_of_unaligned_views(vc, name):
    import torch
    for E, K in ((64, 2), (256, 8), (256, 12), (1024, 8), (40, 3)):
        z, _ = logits(2, 19, E, name, E + K, True)
        dw = put(np.random.default_rng(E).normal(size=(2, 19, K)))
        for normalise in (True, False):
            ids, w = vc.vcoll_moe_route(z, K, normalise=normalise)
            ids2, w2 = vc.vcoll_moe_route(shifted(z), K, normalise=normalise)
            assert torch.equal(ids, ids2) and torch.equal(w, w2), (E, K)
            out = shifted(torch.zeros_like(z), 3)
            vc.vcoll_moe_route_backward(shifted(z), shifted(ids), shifted(w), shifted(dw), normalise=normalise,
                                        d_logits=out)
            assert torch.equal(out, vc.vcoll_moe_route_backward(z, ids, w, dw, normalise=normalise)), (E, K)


def test_route_backward_leaves_out_strange_ids(vc):
    """Slots with ids outside [0, experts) add nothing, whatever their weight and gradient hold."""
    z, z64 = logits(1, 4, 20, "f32", 2, False)
    ids, w = vc.vcoll_moe_route(z, 3)
    for normalise in (True, False):
        bad_ids, bad_w = ids.clone(), w.clone()
        dw = put(np.random.default_rng(3).normal(size=(1, 4, 3)))
        bad_ids[0, 0, 1], bad_ids[0, 1, 0], bad_ids[0, 2] = -7, 20, 2 ** 31 - 1
        gone = (bad_ids < 0) | (bad_ids >= 20)
        if normalise:                                        # what is left of a token is a softmax of its own
            live = put(np.where(get(gone), -np.inf, np.take_along_axis(z64, get(ids).astype(np.int64), 2)))
            bad_w = live.softmax(-1).nan_to_num(0.0)
        else:
            bad_w = vc.vcoll_moe_route(z, 3, normalise=False)[1]
        bad_w[gone] = float("nan")
        dw[gone] = float("inf")
        got = get(vc.vcoll_moe_route_backward(z, bad_ids, bad_w, dw, normalise=normalise)[0])
        want = train.route_backward(z64[0], get(bad_ids[0]), get(dw[0]), normalise)
        size = np.where(get(gone[0]), 0, np.abs(get(dw[0]))).max(axis=1)[:, None]
        close(got, want, (2 * (2 * 50 + 40) + 16) * U * 2 * size + U * np.abs(want), str(normalise))


def test_route_beyond_2_31_logits(vc):
    """The last tokens of a table of more than 2^31 logits."""
    import torch
    T, E = 9_000_000, 250
    z = torch.zeros((1, T, E), device="cuda", dtype=torch.bfloat16)
    tail = torch.randn((40, E), device="cuda").to(torch.bfloat16)
    z[0, -40:] = tail
    ids, w = vc.vcoll_moe_route(z, 3)
    want_ids, want_w = vc.vcoll_moe_route(tail[None].contiguous(), 3)
    assert torch.equal(ids[0, -40:], want_ids[0]) and torch.equal(w[0, -40:], want_w[0])
    assert bool((ids[0, :-40] == torch.arange(3, device="cuda")).all())
    dw = torch.randn((1, T, 3), device="cuda")
    dz = vc.vcoll_moe_route_backward(z, ids, w, dw, normalise=False)
    want = vc.vcoll_moe_route_backward(tail[None].contiguous(), want_ids, want_w, dw[:, -40:].contiguous(),
                                       normalise=False)
    assert torch.equal(dz[0, -40:], want[0])


def test_route_list_and_given_outputs(vc):
    import torch
    z, _ = logits(3, 5, 20, "f32", 1, True)
    ids, w = vc.vcoll_moe_route(z, 4)
    out_i = [torch.full((5, 4), 77, dtype=torch.int32, device="cuda") for _ in range(3)]
    out_w = torch.full((3, 5, 4), 7.0, device="cuda")
    a, b = vc.vcoll_moe_route([z[i].clone() for i in range(3)], 4, ids=out_i, weights=out_w)
    assert a is out_i and b is out_w
    assert all(torch.equal(a[i], ids[i]) and torch.equal(b[i], w[i]) for i in range(3))
    empty = vc.vcoll_moe_route(z[:, :0], 4)
    assert empty[0].shape == (3, 0, 4)
    with pytest.raises(ValueError):
        vc.vcoll_moe_route(z, 4, weights=z.view(-1)[:60].view(3, 5, 4))
    with pytest.raises(vc.VcollError):
        vc.vcoll_moe_route(torch.zeros((1, 2, 1025), device="cuda"), 4)


# --- expert sort ------------------------------------------------------------------

def expert_ids(p, T, K, E, seed, gone=0.2):
    rng = np.random.default_rng(seed)
    w = (np.arange(1, E + 1, dtype=float) ** -1.1)[None, None]
    ids = np.argsort(-(np.log(w) + rng.gumbel(size=(p, T, E))), axis=-1, kind="stable")[..., :K].astype(np.int32)
    ids[rng.random(ids.shape) < gone] = -1
    return ids


SORTS = [(1, 1, 1, 1), (1, 5, 1, 2), (8, 1, 8, 32), (2, 64, 4, 4), (3, 171, 2, 5), (8, 16, 8, 32), (4, 333, 3, 6),
         (2, 700, 5, 512), (1, 1025, 1, 1024), (8, 520, 8, 32), (16, 300, 7, 3), (72, 40, 4, 2), (128, 3, 8, 8)]


@pytest.mark.parametrize("p,T,K,per_rank", SORTS)
def test_sort(vc, p, T, K, per_rank):
    import torch
    ids = expert_ids(p, T, K, p * per_rank, T + K)
    ids[0, 0, 0] = p * per_rank                              # one past the last expert: no expert
    slots, offsets = vc.vcoll_moe_sort(torch.from_numpy(ids).cuda(), per_rank)
    want_slots, want_offsets = train.expert_sort(ids, per_rank)
    assert np.array_equal(get(offsets), want_offsets)
    assert np.array_equal(get(slots), want_slots)


def test_sort_large(vc):
    """More pairs than 256 steps of 1024: tiles of several steps; against a stable argsort."""
    import torch
    p, T, K, per_rank = 8, 9001, 8, 32
    rng = np.random.default_rng(6)
    ids = rng.integers(-1, p * per_rank, (p, T, K)).astype(np.int32)
    slots, offsets = vc.vcoll_moe_sort(torch.from_numpy(ids).cuda(), per_rank)
    key = np.where(ids < 0, p * per_rank, ids).reshape(-1)
    place = np.empty(key.size, np.int64)
    place[np.argsort(key, kind="stable")] = np.arange(key.size)
    counts = np.bincount(key, minlength=p * per_rank + 1)[:-1].reshape(p, per_rank)
    start = np.concatenate([[0], counts.sum(1).cumsum()])
    want = np.stack([np.where(key == p * per_rank, -1, key // per_rank),
                     np.where(key == p * per_rank, -1, place - start[np.minimum(key // per_rank, p)])], -1)
    assert np.array_equal(get(slots).reshape(-1, 2), want)
    assert np.array_equal(get(offsets)[:, 1:], counts.cumsum(1)) and not get(offsets)[:, 0].any()


@pytest.mark.parametrize("ids", ["none", "one", "empty"])
def test_sort_extremes(vc, ids):
    """No pair with an expert, every pair with the same one, no pair at all."""
    import torch
    p, T, K, per_rank = 3, 0 if ids == "empty" else 900, 2, 7
    x = np.full((p, T, K), -1 if ids == "none" else 9, np.int32)
    slots, offsets = vc.vcoll_moe_sort(torch.from_numpy(x).cuda(), per_rank)
    want_slots, want_offsets = train.expert_sort(x, per_rank)
    assert np.array_equal(get(slots), want_slots) and np.array_equal(get(offsets), want_offsets)


def test_sort_given_buffers(vc):
    import torch
    ids = torch.from_numpy(expert_ids(4, 500, 4, 16, 2)).cuda()
    want = vc.vcoll_moe_sort(ids, 4)
    need = vc.vcoll_moe_sort_workspace(4, 500, 4, 4)
    slots = [torch.empty((2000, 2), dtype=torch.int32, device="cuda") for _ in range(4)]
    offsets = torch.empty((4, 5), dtype=torch.int32, device="cuda")
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")        # needs no clearing
    for _ in range(2):
        vc.vcoll_moe_sort([ids[i].clone() for i in range(4)], 4, slots=slots, offsets=offsets, workspace=ws)
        assert torch.equal(torch.stack(slots), want[0]) and torch.equal(offsets, want[1])
    with pytest.raises(vc.VcollError):
        vc.vcoll_moe_sort(ids, 4, workspace=ws[:need - 4])
    with pytest.raises(ValueError):
        vc.vcoll_moe_sort(ids, 4, offsets=want[0].view(-1)[:20].view(4, 5), slots=want[0])


def test_sorted_rows_through_the_dispatch(vc):
    """The dispatch with these slots delivers every expert's rows as one run, in (rank, token, slot) order."""
    import torch
    p, T, K, per_rank, H = 4, 37, 3, 4, 24
    ids = expert_ids(p, T, K, p * per_rank, 8)
    slots, offsets = vc.vcoll_moe_sort(torch.from_numpy(ids).cuda(), per_rank)
    x = torch.randn((p, T, H), device="cuda")
    got = [r.tolist() for r in get(offsets)]
    recv = vc.vcoll_moe_dispatch(list(x), list(slots), [r[-1] for r in got], K)
    for j in range(p):
        for l in range(per_rank):
            at = np.argwhere(ids.reshape(p, -1) == j * per_rank + l)
            want = torch.stack([x[i, n // K] for i, n in at]) if len(at) else x[0, :0]
            assert torch.equal(recv[j][got[j][l]:got[j][l + 1]], want), (j, l)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("H,off", [(1, 0), (3, 0), (8, 0), (24, 0), (72, 1), (144, 0), (500, 0), (1001, 0), (1024, 0),
                                   (1032, 3), (2639, 0), (4096, 0), (4100, 1)])
def test_dispatch_rows_of_any_width(vc, name, H, off):
    """Short, odd and unaligned rows (the last receive rows untouched): the same bytes as indexing."""
    import torch
    p, T, K, per_rank = 3, 21, 5, 4
    ids = expert_ids(p, T, K, p * per_rank, H)
    slots, offsets = train.expert_sort(ids, per_rank)

    def flat(n):
        return torch.full((n + off,), 7.0, device="cuda", dtype=dt(name))[off:]
    x = [flat(T * H).view(T, H).copy_(torch.randn((T, H), device="cuda")) for _ in range(p)]
    rows = [int(offsets[j, -1]) for j in range(p)]
    recv = [flat((n + 1) * H).view(n + 1, H) for n in rows]
    vc.vcoll_moe_dispatch(x, [put_ids(s) for s in slots], rows, K, recv=recv)
    for i in range(p):
        for n, (j, r) in enumerate(slots[i]):
            if j >= 0:
                assert torch.equal(recv[j][r], x[i][n // K]), (i, n)
    assert all(bool((recv[j][rows[j]] == 7).all()) for j in range(p))


# --- weighted combine ---------------------------------------------------------------

def experts_case(p, T, K, H, per_rank, name, seed, gone=0.2, spare=2):
    """Slots of a dispatch with some pairs missing, and expert rows (a few more than are named)."""
    ids = expert_ids(p, T, K, p * per_rank, seed, gone)
    slots, offsets = train.expert_sort(ids, per_rank)
    rng = np.random.default_rng(seed + 1)
    e = [put(rng.normal(size=(int(offsets[j, -1]) + spare, H)), name) for j in range(p)]
    w = put(rng.normal(size=(p, T, K)))
    return put_ids(slots), slots, e, w, rng


def put_ids(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


COMBINES = [(1, 1, 1, 1, 1, "f32"), (1, 1, 8, 7168, 8, "bf16"), (2, 5, 2, 16, 3, "bf16"), (3, 9, 3, 1001, 2, "f32"),
            (3, 9, 3, 1001, 2, "bf16"), (8, 4, 8, 512, 32, "bf16"), (2, 3, 9, 260, 8, "f32"), (1, 2, 17, 4096, 20, "bf16"),
            (1, 3, 4, 9000, 6, "bf16"), (4, 6, 2, 2056, 2, "f32"), (40, 2, 2, 64, 1, "f32"), (2, 4, 33, 40, 20, "bf16"), (1, 3, 70, 24, 80, "f32"), (1, 2, 62, 16, 64, "bf16"),
            (1, 2, 130, 9, 132, "f32"),
            (2, 7, 5, 8, 4, "bf16"), (2, 7, 1, 3, 4, "bf16")]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("p,T,K,H,per_rank,name", COMBINES)
def test_combine_weighted(vc, p, T, K, H, per_rank, name, weighted):
    ts, slots, e, w, _ = experts_case(p, T, K, H, per_rank, name, T * K + H)
    out = vc.vcoll_moe_combine_weighted(e, ts, w if weighted else None, T, K)
    want, size = train.combine_weighted([get(x) for x in e], slots, get(w) if weighted else None, T, K)
    # K products and K additions, then one rounding to the storage type
    close(get(out), want, (K + 1) * U * size + half_step(name) * np.abs(want) + 2.0 ** -126, "out")


@pytest.mark.parametrize("p,T,K,H,per_rank,name", COMBINES)
def test_combine_weighted_backward(vc, p, T, K, H, per_rank, name):
    ts, slots, e, w, rng = experts_case(p, T, K, H, per_rank, name, T * K + H + 1)
    dy = put(rng.normal(size=(p, T, H)), name)
    mine = [x.new_full(x.shape, 7.0) for x in e]
    de, dw = vc.vcoll_moe_combine_weighted_backward(dy, e, ts, w, K, d_expert_out=mine)
    want_de, want_dw, size = train.combine_weighted_backward(get(dy), [get(x) for x in e], slots, get(w), K)
    # products along a chain of at most H / 64 + 32 additions on any lane, then one over lanes
    close(get(dw), want_dw, (H / 64 + 64) * U * size, "d_weights")
    for j in range(p):
        left = np.isnan(want_de[j])
        assert (get(de[j])[left] == 7.0).all(), "rows without a slot"
        want = np.where(left, 7.0, want_de[j])
        close(get(de[j]), want, (U + half_step(name)) * (1 + U) * np.abs(want), f"d_expert {j}")
    made, dw2 = vc.vcoll_moe_combine_weighted_backward(dy, e, ts, w, K)
    assert (get(dw2) == get(dw)).all()
    assert all((get(made[j]) == np.where(np.isnan(want_de[j]), 0, get(de[j]))).all() for j in range(p))


def test_combine_gradient_against_differences(vc):
    """out is linear in each argument: a finite difference of the forward pass is the gradient, up to its rounding."""
    p, T, K, H = 2, 3, 2, 8
    ts, slots, e, w, rng = experts_case(p, T, K, H, 3, "f32", 5)
    dy = put(rng.normal(size=(p, T, H)))
    de, dw = vc.vcoll_moe_combine_weighted_backward(dy, e, ts, w, K)
    base = get(vc.vcoll_moe_combine_weighted(e, ts, w, T, K))
    for i, t, k in np.ndindex(p, T, K):
        w2 = w.clone()
        w2[i, t, k] += 1.0
        num = ((get(vc.vcoll_moe_combine_weighted(e, ts, w2, T, K)) - base) * get(dy)).sum()
        assert abs(num - float(dw[i, t, k])) < 2 * (K + 3) * U * 8 * H * 16          # |out| < 8, |dy| < 4
    for j in range(p):
        for r in range(e[j].shape[0]):
            e2 = [x.clone() for x in e]
            e2[j][r] += 1.0
            num = ((get(vc.vcoll_moe_combine_weighted(e2, ts, w, T, K)) - base) * get(dy)).sum()
            assert abs(num - float(de[j][r].sum())) < 2 * (K + 3) * U * 8 * H * 16


def test_combine_skips_what_slots_do_not_name(vc):
    """Infinities and NaN in unnamed rows and in the weights of missing pairs reach nothing; a token without slots gets
    zeros; slots out of range in either part are skipped."""
    import torch
    p, T, K, H = 2, 4, 2, 40
    for name in ("f32", "bf16"):
        e = [torch.ones((3, H), device="cuda", dtype=dt(name)) for _ in range(p)]
        e[0][2] = float("nan")
        e[1][0] = float("inf")
        s = np.full((p, T * K, 2), -1, np.int32)
        s[0, 0], s[0, 2], s[0, 3], s[0, 5] = (0, 0), (2, 0), (-7, 1), (0, 3)
        s[1, 1], s[1, 7] = (1, 2), (1, -1)
        w = torch.full((p, T, K), float("nan"), device="cuda")
        w[0, 0, 0], w[1, 0, 1] = 2.0, 3.0
        out = get(vc.vcoll_moe_combine_weighted(e, put_ids(s), w, T, K))
        assert (out[0, 0] == 2).all() and (out[1, 0] == 3).all() and not out[:, 1:].any()
        de, dw = vc.vcoll_moe_combine_weighted_backward(torch.ones((p, T, H), device="cuda", dtype=dt(name)), e,
                                                        put_ids(s), w, K)
        assert (get(de[0])[0] == 2).all() and (get(de[1])[2] == 3).all()
        assert not get(de[0])[1:].any() and not get(de[1])[:2].any()
        want = np.zeros((p, T, K))
        want[0, 0, 0] = want[1, 0, 1] = H
        assert np.array_equal(get(dw), want)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_combine_of_unaligned_views(vc, name):
    """Buffers one element off a 16-byte boundary: same results."""
    import torch
    p, T, K, H = 2, 5, 3, 264
    ts, slots, e, w, rng = experts_case(p, T, K, H, 3, name, 9)
    dy = put(rng.normal(size=(p, T, H)), name)

    def shift(x):
        flat = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        y = flat[1:].view(x.shape)
        y.copy_(x)
        return y
    a = vc.vcoll_moe_combine_weighted(e, ts, w, T, K)
    b = vc.vcoll_moe_combine_weighted([shift(x) for x in e], ts, w, T, K)
    assert torch.equal(a, b)
    de, dw = vc.vcoll_moe_combine_weighted_backward(dy, e, ts, w, K)
    de2, dw2 = vc.vcoll_moe_combine_weighted_backward(shift(dy), [shift(x) for x in e], ts, w, K,
                                                      d_expert_out=[shift(torch.zeros_like(x)) for x in e])
    assert all(torch.equal(x, y) for x, y in zip(de, de2))
    _, want, size = train.combine_weighted_backward(get(dy), [get(x) for x in e], slots, get(w), K)
    close(get(dw2), want, (H / 64 + 64) * U * size, "d_weights")


def test_combine_of_lists_and_given_outputs(vc):
    """Rank buffers as lists, results into given buffers; the refusals of overlaps."""
    import torch
    p, T, K, H = 3, 6, 3, 72
    ts, slots, e, w, rng = experts_case(p, T, K, H, 2, "bf16", 6)
    dy = put(rng.normal(size=(p, T, H)), "bf16")
    want = vc.vcoll_moe_combine_weighted(e, ts, w, T, K)
    want_e, want_w = vc.vcoll_moe_combine_weighted_backward(dy, e, ts, w, K)
    lists = lambda x: [x[i].clone() for i in range(p)]                                        # noqa: E731
    out = [torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(p)]
    assert vc.vcoll_moe_combine_weighted(e, lists(ts), lists(w), T, K, out=out) is out
    assert torch.equal(torch.stack(out), want)
    dw = torch.full((p, T, K), 7.0, device="cuda")
    de, dw2 = vc.vcoll_moe_combine_weighted_backward(lists(dy), e, lists(ts), lists(w), K, d_weights=dw)
    assert dw2 is dw and torch.equal(dw, want_w) and all(torch.equal(a, b) for a, b in zip(de, want_e))
    assert isinstance(vc.vcoll_moe_combine_weighted(e, lists(ts), w, T, K), list)
    with pytest.raises(ValueError):
        vc.vcoll_moe_combine_weighted_backward(dy, e, ts, w, K, d_expert_out=e)
    with pytest.raises(ValueError):
        vc.vcoll_moe_combine_weighted_backward(dy, e, ts, w, K, d_expert_out=[e[0][:1]] * p)
    with pytest.raises(ValueError):
        vc.vcoll_moe_combine_weighted_backward(dy, e, ts, w, K, d_weights=w)
    with pytest.raises(ValueError):
        vc.vcoll_moe_combine_weighted([dy[i] for i in range(p)], ts, w, T, K, out=dy)
    empty = vc.vcoll_moe_combine_weighted([x[:0] for x in e], ts, w, T, K)
    assert not bool(empty.any()), "no expert row at all: zeros"
    none = vc.vcoll_moe_combine_weighted(e, ts[:, :0].contiguous(), w[:, :0].contiguous(), 0, K)
    assert none.shape == (p, 0, H)


def test_combine_rows_beyond_4_gib(vc):
    """Byte offsets past 2^32 inside one expert buffer."""
    import torch
    H, R = 7168, 320_000                                     # 4.6 GB of bf16
    e = torch.empty((R, H), dtype=torch.bfloat16, device="cuda")
    e[0] = 1.0
    e[R - 1] = 2.0
    s = put_ids(np.array([[[0, R - 1], [0, 0]]], np.int32))
    w = put(np.array([[[0.5, 0.25]]]))
    assert (get(vc.vcoll_moe_combine_weighted([e], s, w, 1, 2)) == 1.25).all()
    dy = torch.full((1, 1, H), 4.0, dtype=torch.bfloat16, device="cuda")
    de = torch.empty_like(e)
    _, dw = vc.vcoll_moe_combine_weighted_backward(dy, [e], s, w, 2, d_expert_out=[de])
    assert get(dw).tolist() == [[[2 * 4 * H, 4 * H]]]
    assert (get(de[R - 1]) == 2).all() and (get(de[0]) == 1).all()


def test_combine_reverses_the_dispatch(vc):
    """With weights that add up to 1 per token the combine of dispatched rows gives the tokens back; its gradient with
    ones gives K times."""
    import torch
    p, T, K, H, per_rank = 4, 50, 4, 128, 4
    x = torch.randn((p, T, H), device="cuda")
    ids, w = vc.vcoll_moe_route(torch.randn((p, T, p * per_rank), device="cuda"), K)
    slots, offsets = vc.vcoll_moe_sort(ids, per_rank)
    recv = vc.vcoll_moe_dispatch(list(x), list(slots), offsets[:, -1].tolist(), K)
    back = get(vc.vcoll_moe_combine_weighted(recv, slots, w, T, K))
    # the weights add up to 1 within (2 * 20 + 40) u each; K products and additions
    close(back, get(x), (2 * 20 + 40 + 2 * K + 1) * U * np.abs(get(x)), "tokens")
    ones = get(vc.vcoll_moe_combine_weighted(recv, slots, None, T, K))
    assert np.array_equal(ones, K * get(x))                  # 4 x is exact, and so are 2 x and 3 x rounded alike


# --- AdamW --------------------------------------------------------------------------

HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, grad_scale=0.5)
SIZES = [1, 7, 128, 129, 2047, 2048, 2049, 5000, 0, 3, 20000]


def adam_inputs(name, grad, bits, sizes, seed, off=0):
    """Tensors that start `off` elements into their own allocation, with states after some training."""
    import torch
    rng = np.random.default_rng(seed)

    def view(x, d):
        flat = torch.zeros(x.size + off, dtype=d, device="cuda")
        flat[off:].copy_(torch.from_numpy(x))
        return flat[off:]
    host, dev = [], {k: [] for k in ("params", "grads", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale",
                                     "master")}
    for k, n in enumerate(sizes):
        x = (rng.normal(size=n) * 0.1).astype(np.float32)
        g = view((rng.normal(size=n) * 10.0 ** rng.integers(-6, 1, n)).astype(np.float32), dt(grad))
        m = (rng.normal(size=n) * 1e-3).astype(np.float32)
        v = (rng.normal(size=n) ** 2 * 1e-6).astype(np.float32)
        v[::5] = 0
        h = dict(x=x, g=g.float().cpu().numpy(), m=m, v=v)
        if bits == 8:
            b = train.rounding_bits(n, 1, 0, k)
            for s, enc, dec in (("m", train.encode_m, train.decode_m), ("v", train.encode_v, train.decode_v)):
                code, scale = enc(h[s], b)
                h[s] = dec(code, scale)
                dev["exp_avg" if s == "m" else "exp_avg_sq"].append(view(code, torch.uint8))
                dev["exp_avg_scale" if s == "m" else "exp_avg_sq_scale"].append(torch.from_numpy(scale).cuda())
        else:
            dev["exp_avg"].append(view(m, torch.float32))
            dev["exp_avg_sq"].append(view(v, torch.float32))
        dev["grads"].append(g)
        dev["params"].append(view(x, dt(name)))
        dev["master"].append(view(x, torch.float32))
        host.append(h)
    if name == "f32":
        del dev["master"]
    if bits == 32:
        del dev["exp_avg_scale"], dev["exp_avg_sq_scale"]
    return host, dev


def same_bits(t, want, what):
    got = t.cpu().numpy()
    view = {4: np.uint32, 1: np.uint8}[got.itemsize]
    bad = (got.view(view) != want.astype(got.dtype).view(view)) & ~(np.isnan(want) & np.isnan(got.astype(np.float64)))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} differ, first {np.flatnonzero(bad)[:3]}: " \
                          f"{got[bad][:3]} want {want[bad][:3]}"


@pytest.mark.parametrize("off", [0, 1, 3])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_adamw(vc, name, grad, bits, off):
    """Three steps over tensors of many sizes, bit for bit."""
    import torch
    host, dev = adam_inputs(name, grad, bits, SIZES, 11 + off, off)
    run = vc.prepare_adamw(**dev)
    for step in (1, 2, 3):
        run(step=step, seed=5, **HYPER)
        for k, h in enumerate(host):
            h["x"], h["m"], h["v"] = train.adamw(h["x"], h["g"], h["m"], h["v"], step=step, **HYPER)
            at = f"step {step} tensor {k}"
            same_bits(dev["master" if name == "bf16" else "params"][k], h["x"], at + " parameters")
            if name == "bf16":
                assert torch.equal(dev["params"][k], dev["master"][k].to(torch.bfloat16)), at
            if bits == 32:
                same_bits(dev["exp_avg"][k], h["m"], at + " exp_avg")
                same_bits(dev["exp_avg_sq"][k], h["v"], at + " exp_avg_sq")
                continue
            b = train.rounding_bits(h["m"].size, 5, step, k)
            for s, state, enc, dec in (("m", "exp_avg", train.encode_m, train.decode_m),
                                       ("v", "exp_avg_sq", train.encode_v, train.decode_v)):
                code, scale = enc(h[s], b)
                same_bits(dev[state][k], code, f"{at} {state} codes")
                same_bits(dev[state + "_scale"][k], scale, f"{at} {state} scales")
                h[s] = dec(code, scale)


def test_adamw_many_tensors(vc):
    """More tensors than one launch describes."""
    sizes = [1 + 97 * k % 400 for k in range(150)]
    for bits in (32, 8):
        host, dev = adam_inputs("f32", "f32", bits, sizes, 2)
        vc.vcoll_adamw(dev.pop("params"), dev.pop("grads"), dev["exp_avg"], dev["exp_avg_sq"], step=4, seed=9,
                       exp_avg_scale=dev.get("exp_avg_scale"), exp_avg_sq_scale=dev.get("exp_avg_sq_scale"), **HYPER)
        for k, h in enumerate(host):
            _, m, v = train.adamw(h["x"], h["g"], h["m"], h["v"], step=4, **HYPER)
            if bits == 8:
                b = train.rounding_bits(m.size, 9, 4, k)
                m, v = train.encode_m(m, b)[0], train.encode_v(v, b)[0]
            same_bits(dev["exp_avg"][k], m, f"tensor {k}")
            same_bits(dev["exp_avg_sq"][k], v, f"tensor {k}")


def test_adamw_beyond_2_32_elements(vc):
    """The last 1500 elements of a tensor of 2^32 + 1500 with 8-bit states: offsets and random bits past 32 bits."""
    import torch
    n, m = 2 ** 32 + 1500, 1500
    x = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    state = vc.adamw_state([x], 8)
    rng = np.random.default_rng(8)
    xs = (rng.normal(size=m) * 0.1).astype(np.float32)
    x[-m:].copy_(torch.from_numpy(xs))
    g[-m:].copy_(torch.from_numpy((rng.normal(size=m) * 1e-3).astype(np.float32)))
    gs = g[-m:].float().cpu().numpy()
    vc.vcoll_adamw([x], [g], **state, step=1, seed=4, **HYPER)
    z = np.zeros(m, np.float32)
    want, wm, wv = train.adamw(xs, gs, z, z, step=1, **HYPER)
    b = train.rounding_bits(m, 4, 1, 0, 2 ** 32)
    same_bits(x[-m:], want, "parameters")
    same_bits(state["exp_avg"][0][-m:], train.encode_m(wm, b)[0], "exp_avg")
    same_bits(state["exp_avg_sq"][0][-m:], train.encode_v(wv, b)[0], "exp_avg_sq")
    assert not bool(x[:-m].any()) and not bool(state["exp_avg"][0][:-m].any())


def test_adamw_from_zero_states(vc):
    import torch
    for name in ("f32", "bf16"):
        for bits in (32, 8):
            x = [torch.randn(300, device="cuda").to(dt(name))]
            g = [torch.randn(300, device="cuda")]
            state = vc.adamw_state(x, bits)
            was = x[0].float().cpu().numpy()
            vc.vcoll_adamw(x, g, **state, step=1, **HYPER)
            z = np.zeros(300, np.float32)
            want, _, _ = train.adamw(was, g[0].cpu().numpy(), z, z, step=1, **HYPER)
            same_bits(state["master"][0] if name == "bf16" else x[0], want, f"{name} {bits}")


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_values_at_the_edges(vc, bits):
    """NaN, infinities, overflow of g^2 and denormals, in groups with ordinary values beside them."""
    import torch
    g = np.full(512, 1e-3, np.float32)
    g[3], g[130], g[131], g[200] = np.nan, np.inf, -np.inf, 1e30
    g[256:384] = 1e-42
    g[384:] = 0
    x = np.linspace(-1, 1, 512, dtype=np.float32)
    z = np.zeros(512, np.float32)
    p = [torch.from_numpy(x).cuda()]
    state = vc.adamw_state(p, bits)
    vc.vcoll_adamw(p, [torch.from_numpy(g).cuda()], **state, step=1, seed=3, **HYPER)
    with np.errstate(all="ignore"):
        want, m, v = train.adamw(x, g, z, z, step=1, **HYPER)
        same_bits(p[0], want, "parameters")
        if bits == 8:
            b = train.rounding_bits(512, 3, 1, 0)
            for t, s, enc, y in (("exp_avg", "exp_avg_scale", train.encode_m, m),
                                 ("exp_avg_sq", "exp_avg_sq_scale", train.encode_v, v)):
                code, scale = enc(y, b)
                same_bits(state[t][0], code, t)
                same_bits(state[s][0], scale, s)
        else:
            same_bits(state["exp_avg"][0], m, "exp_avg")
            same_bits(state["exp_avg_sq"][0], v, "exp_avg_sq")


def test_unpack(vc):
    """Every code of both formats at several scales; odd lengths and offsets."""
    import torch
    codes = np.tile(np.arange(256, dtype=np.uint8), 3)[:701]
    sm = np.exp2(np.array([0, 3, -20, 100, -126, 1])).astype(np.float32)
    sv = np.exp2(np.array([5, -9, 0, 126, -90, 2])).astype(np.float32)
    for off in (0, 1, 5):
        flat = torch.zeros(codes.size + off, dtype=torch.uint8, device="cuda")
        flat[off:].copy_(torch.from_numpy(codes))
        m, v = vc.vcoll_adamw_unpack(flat[off:], flat[off:].clone(), put(sm), put(sv))
        same_bits(m, train.decode_m(codes, sm), "exp_avg")
        same_bits(v, train.decode_v(codes, sv), "exp_avg_sq")


def test_adamw_refuses_overlap(vc):
    import torch
    x = torch.zeros(16, device="cuda")
    y, z = torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")
    with pytest.raises(ValueError):
        vc.vcoll_adamw([x[:8]], [x[8:]], [y], [x[4:12]], lr=1.0, step=1)
    with pytest.raises(ValueError):
        vc.vcoll_adamw([x[:8]], [x[4:12]], [y], [z], lr=1.0, step=1)


# --- all of them ----------------------------------------------------------------------

def whole_step(vc, s):
    ids, w = vc.vcoll_moe_route(s["z"], s["K"], ids=s["ids"], weights=s["w"])
    slots, offsets = vc.vcoll_moe_sort(ids, s["per_rank"], slots=s["slots"], offsets=s["offsets"], workspace=s["ws"])
    vc.vcoll_moe_dispatch(list(s["x"]), list(slots), [r.shape[0] for r in s["recv"]], s["K"], recv=s["recv"])
    y = vc.vcoll_moe_combine_weighted(s["recv"], slots, w, s["T"], s["K"], out=s["y"])
    vc.vcoll_moe_combine_weighted_backward(y, s["recv"], slots, w, s["K"], d_expert_out=s["de"], d_weights=s["dw"])
    vc.vcoll_moe_route_backward(s["z"], ids, w, s["dw"], d_logits=s["dz"])
    vc.vcoll_moe_combine_weighted(s["de"], slots, None, s["T"], s["K"], out=s["dx"])


def step_buffers(vc, seed):
    import torch
    p, T, K, per_rank, H = 4, 200, 4, 8, 256
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *sh, d=torch.float32: torch.full(sh, 3, dtype=d, device="cuda")              # noqa: E731
    s = dict(T=T, K=K, per_rank=per_rank, z=torch.randn((p, T, p * per_rank), device="cuda", generator=g),
             x=torch.randn((p, T, H), device="cuda", generator=g).bfloat16())
    s.update(ids=new(p, T, K, d=torch.int32), w=new(p, T, K), slots=new(p, T * K, 2, d=torch.int32),
             offsets=new(p, per_rank + 1, d=torch.int32), y=new(p, T, H, d=torch.bfloat16), dw=new(p, T, K),
             dz=new(p, T, p * per_rank), dx=new(p, T, H, d=torch.bfloat16),
             ws=new(vc.vcoll_moe_sort_workspace(p, T, K, per_rank), d=torch.uint8),
             recv=[new(2 * T * K, H, d=torch.bfloat16) for _ in range(p)],
             de=[new(2 * T * K, H, d=torch.bfloat16) for _ in range(p)])
    return s


def snapshot(s):
    import torch
    names = ("ids", "w", "slots", "offsets", "y", "dw", "dz", "dx")
    return [s[k].clone() for k in names] + [t.clone() for t in s["recv"] + s["de"]] + [torch.zeros(1)]


def test_captured_step_replays(vc):
    """The whole step, without a copy to the host, captured and replayed on changing inputs."""
    import torch
    s = step_buffers(vc, 31)
    whole_step(vc, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        whole_step(vc, s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("capturing")
    with torch.cuda.graph(graph):
        whole_step(vc, s)
    for rep in range(4):
        s["z"].copy_(torch.randn_like(s["z"]))
        s["x"].copy_(torch.randn_like(s["z"])[..., :1].expand_as(s["x"]))
        whole_step(vc, s)
        torch.cuda.synchronize()
        want = snapshot(s)
        for t in (s["ids"], s["w"], s["slots"], s["offsets"], s["y"], s["dw"], s["dz"], s["dx"], s["ws"]):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(snapshot(s), want)), rep


def test_captured_adamw_replays(vc):
    import torch
    x = [torch.randn(5000, device="cuda"), torch.randn(77, device="cuda")]
    for bits in (32, 8):
        params = [t.clone() for t in x]
        grads = [torch.randn_like(t) for t in x]
        state = vc.adamw_state(params, bits)
        run = vc.prepare_adamw(params, grads, **state)
        keep = [params] + list(state.values())
        zero = [[t.clone() for t in ts] for ts in keep]
        run(step=2, seed=1, **HYPER)
        torch.cuda.synchronize()
        want = [[t.clone() for t in ts] for ts in keep]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(step=2, seed=1, **HYPER)
        for rep in range(3):
            for ts, zs in zip(keep, zero):
                for t, z in zip(ts, zs):
                    t.copy_(z)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for ts, ws in zip(keep, want) for a, b in zip(ts, ws)), (bits, rep)


def test_on_another_stream(vc):
    """Calls follow torch's current stream: on a side stream behind a long fill, results are those of the main one."""
    import torch
    s = step_buffers(vc, 32)
    whole_step(vc, s)
    torch.cuda.synchronize()
    want = snapshot(s)
    t = step_buffers(vc, 33)
    z, x = s["z"], s["x"]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.zeros(1 << 28, device="cuda")
        for _ in range(4):
            big.add_(1.0)
        t["z"].copy_(z)
        t["x"].copy_(x)
        whole_step(vc, t)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(snapshot(t), want))


def test_results_repeat(vc):
    """Same inputs, same bits, whatever the order of workgroups."""
    import torch
    s = step_buffers(vc, 34)
    whole_step(vc, s)
    want = snapshot(s)
    for _ in range(5):
        whole_step(vc, s)
        assert all(torch.equal(a, b) for a, b in zip(snapshot(s), want))
