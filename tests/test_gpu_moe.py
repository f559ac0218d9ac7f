"""GPU parity of the mixture-of-experts operators with the fp64 oracle (oracle/moe.py)."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tile_level_sync_gb300 as cs
from oracle import moe as ref
from moe_helpers import assert_within, f64, layer, mlp_inputs, run_mlp, run_mlp_grad

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 2, 2), (33, 7, 3), (500, 60, 8), (513, 1024, 8),
                                   (2000, 5, 2), (2049, 37, 2), (9000, 256, 3), (70000, 33, 9)])
@pytest.mark.parametrize("how", ["random", "one", "invalid"])
def test_plan(T, E, k, how):
    rng = np.random.default_rng(T + E + k)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if how == "one":
        ids[:] = E - 1
    if how == "invalid":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E + 3
        ids[rng.random((T, k)) < 0.05] = -(1 << 31)
    m = cs.Moe(cs.make_moe_desc(T=T, experts=E, top_k=min(k, E)) if k <= E else
               cs.make_moe_desc(T=T * k, experts=E, top_k=1))
    if k > E:
        ids = ids.reshape(T * k, 1)
    buf = torch.full((m.info.plan_bytes // 4 + 64,), 12345, dtype=torch.int32, device="cuda")
    plan = buf[:-64]
    m.plan(torch.from_numpy(ids).cuda(), plan)
    want = ref.plan(ids, E)
    for name, got in m.plan_views(plan).items():
        assert np.array_equal(got.cpu().numpy(), want[name]), name
    assert bool((buf[-64:] == 12345).all())
    assert m.check(plan) == (cs.OK, 0)


# ------------------------------------------------------------------ route

ROUTES = [
    dict(T=1, E=64, k=8, score="softmax", renorm=True),
    dict(T=3, E=1, k=1, score="sigmoid"),
    dict(T=77, E=60, k=4, score="softmax"),
    dict(T=77, E=33, k=4, score="softmax", bias=True, renorm=True, scale=2.5),
    dict(T=50, E=256, k=8, score="sigmoid", bias=True, groups=8, group_limit=4, group_top=2, renorm=True, scale=2.5),
    dict(T=50, E=160, k=6, score="softmax", groups=8, group_limit=3, group_top=1, scale=16.0),
    dict(T=40, E=96, k=6, score="softmax", groups=32, group_limit=5, group_top=2, bias=True),
    dict(T=9, E=1024, k=32, score="sigmoid", renorm=True),
    dict(T=9, E=1000, k=32, score="softmax", bias=True, groups=4, group_limit=1, group_top=2),
    dict(T=20, E=8, k=8, score="softmax", renorm=True),
    dict(T=30, E=64, k=6, score="sigmoid", groups=8, group_limit=2, group_top=1, renorm=True),
    dict(T=30, E=128, k=4, score="softmax", groups=4, group_limit=2, group_top=2),
    dict(T=30, E=255, k=20, score="sigmoid", bias=True),
    dict(T=5000, E=32, k=2, score="sigmoid", bias=True, groups=4, group_limit=1, group_top=2, renorm=True),
    dict(T=20, E=8, k=4, score="sigmoid", groups=8, group_limit=4, group_top=2),
]


def _route_case(c, f32, mask, seed=0):
    rng = np.random.default_rng(seed + c["T"] * 1000 + c["E"])
    logits = torch.from_numpy(rng.normal(0, 1.5, (c["T"], c["E"])).astype(np.float32))
    if mask == "some":
        logits[torch.from_numpy(rng.random((c["T"], c["E"])) < 0.5)] = float("-inf")
        logits[torch.from_numpy(rng.random((c["T"], c["E"])) < 0.05)] = float("nan")
        logits[0] = float("-inf")
    elif mask == "lowest":
        logits[torch.from_numpy(rng.random((c["T"], c["E"])) < 0.9)] = torch.finfo(torch.bfloat16).min
    elif mask == "equal":
        logits[:] = logits[:, :1]
    logits = logits if f32 else logits.to(torch.bfloat16)
    bias = torch.from_numpy(rng.normal(0, 0.1, c["E"]).astype(np.float32)) if c.get("bias") else None
    if mask == "equal" and bias is not None:
        bias[:] = 0.25
    return logits, bias


def _layer(c, f32):
    return cs.Moe(cs.make_moe_desc(T=c["T"], experts=c["E"], top_k=c["k"], score=c["score"], groups=c.get("groups", 1),
                                   group_limit=c.get("group_limit", 0), group_top=c.get("group_top", 1),
                                   renorm=c.get("renorm", False), scale=c.get("scale", 1.0), logits_f32=f32))


def _oracle_route(c, logits, bias):
    return ref.route(f64(logits), None if bias is None else f64(bias), c["k"], c["score"], c.get("groups", 1),
                     c.get("group_limit", 0), c.get("group_top", 1), c.get("renorm", False), c.get("scale", 1.0))


def _run_route(c, logits, bias, f32):
    m = _layer(c, f32)
    ids = torch.full((c["T"], c["k"]), 77, dtype=torch.int32, device="cuda")
    w = torch.full((c["T"], c["k"]), float("nan"), device="cuda")
    m.route(logits.cuda(), None if bias is None else bias.cuda(), ids, w)
    return ids.cpu().numpy(), f64(w)


# An fp32 weight: the exponential (2 ulp), its argument's rounding (|l - max| <= 200 where the
# weight is not negligible: below, 200 steps), sums of at most 1024 terms in 37 additions,
# a division and a product: 2^-24 * (2 * 2 + 200 + 37 + 2) < 2^-16 of the value.
ROUTE_TOL = 2.0 ** -16


@pytest.mark.parametrize("c", ROUTES, ids=lambda c: f"T{c['T']}E{c['E']}k{c['k']}{c['score']}")
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("mask", ["none", "some", "lowest", "equal"])
def test_route(c, f32, mask):
    logits, bias = _route_case(c, f32, mask)
    want_ids, want_w = _oracle_route(c, logits, bias)
    ids, w = _run_route(c, logits, bias, f32)
    assert np.array_equal(ids, want_ids)
    assert np.all(np.abs(w - want_w) <= ROUTE_TOL * np.abs(want_w) + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_near_ties(score, groups):
    """Keys that differ in the tenth digit: biases that undo the scores' differences but for
    1e-10, which 32-bit keys cannot see."""
    T, E, k = 64, 64, 8
    rng = np.random.default_rng(3)
    bias = np.float32(rng.choice([0.5, 0.25, 0.125], E))
    logits = np.zeros((T, E), np.float32)
    for t in range(T):
        # one value in an expert's logit, a neighbour 2^-24 away in relative terms
        base = np.float32(rng.normal())
        logits[t] = base * (1 + np.float32(2.0 ** -23) * rng.integers(0, 4, E)).astype(np.float32)
    c = dict(T=T, E=E, k=k, score=score, bias=True, groups=groups, group_limit=min(2, groups), group_top=2)
    want_ids, _ = _oracle_route(c, torch.from_numpy(logits), torch.from_numpy(bias))
    ids, _ = _run_route(c, torch.from_numpy(logits), torch.from_numpy(bias), True)
    assert np.array_equal(ids, want_ids)


@pytest.mark.parametrize("c", [c for c in ROUTES if c["T"] > 1], ids=lambda c: f"T{c['T']}E{c['E']}k{c['k']}{c['score']}")
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("mask", ["none", "some"])
def test_route_grad(c, f32, mask):
    logits, bias = _route_case(c, f32, mask)
    ids, _ = _oracle_route(c, logits, bias)
    dw = np.random.default_rng(1).normal(size=ids.shape).astype(np.float32)
    m = _layer(c, f32)
    dl = torch.full_like(logits, 77).cuda()
    m.route_grad(logits.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), dl)
    renorm, scale = c.get("renorm", False), c.get("scale", 1.0)
    want = ref.route_grad(f64(logits), ids, dw.astype(np.float64), c["score"], renorm, scale)
    # the gradient is a difference of terms of size scale * |dw|_max * s / (1 or sum s)
    size = scale * np.abs(dw).max(axis=1, keepdims=True)
    s = ref.scores(f64(logits), c["score"])
    if renorm:
        total = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0).sum(axis=1, keepdims=True)
        s = np.divide(s, total, out=np.zeros_like(s), where=total > 0)
    half = 0.0 if f32 else ref.BF16
    assert np.all(np.abs(f64(dl) - want) <= 2 * ROUTE_TOL * size * s + half * np.abs(want) + 1e-37)


@pytest.mark.parametrize("E", [64, 33])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", False)])
def test_route_grad_of_an_expert_given_twice(E, score, renorm):
    c = dict(T=37, E=E, k=6, score=score, renorm=renorm)
    logits, _ = _route_case(c, True, "none")
    ids, _ = _oracle_route(c, logits, None)
    ids[::2, 3], ids[::3, 5], ids[5] = ids[::2, 0], E, -1
    dw = np.random.default_rng(1).normal(size=ids.shape).astype(np.float32)
    dl = torch.full_like(logits, 77).cuda()
    _layer(c, True).route_grad(logits.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), dl)
    ids[ids == E] = -1
    want = ref.route_grad(f64(logits), ids, dw.astype(np.float64), score, renorm, 1.0)
    assert np.all(np.abs(f64(dl) - want) <= 4 * ROUTE_TOL * np.abs(dw).max())


def test_route_grad_against_differences():
    c = dict(T=6, E=40, k=5, score="softmax")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            c = dict(T=6, E=40, k=5, score=score, renorm=renorm, scale=1.5)
            logits, _ = _route_case(c, True, "none", seed=5)
            ids, _ = _run_route(c, logits, None, True)
            dw = np.random.default_rng(2).normal(size=ids.shape).astype(np.float32)
            dl = torch.empty_like(logits, device="cuda")
            _layer(c, True).route_grad(logits.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), dl)
            l, h = f64(logits), 1e-5
            for e in range(c["E"]):
                up, down = l.copy(), l.copy()
                up[:, e] += h
                down[:, e] -= h
                f = [(ref.route_weights(x, ids, score, renorm, 1.5) * dw).sum(axis=1) for x in (up, down)]
                # central differences: h^2 times a third derivative below 10, and 1e-16 / h
                assert np.all(np.abs(f64(dl)[:, e] - (f[0] - f[1]) / (2 * h)) <= 2e-5)


# ------------------------------------------------------------------ mlp and its gradient

MLPS = [
    dict(T=1, E=8, k=2, D=64, N1=64),
    dict(T=1, E=3, k=3, D=8, N1=8),
    dict(T=4, E=16, k=8, D=264, N1=136),
    dict(T=33, E=4, k=1, D=64, N1=64),
    dict(T=40, E=4, k=2, D=72, N1=40),
    dict(T=37, E=9, k=3, D=328, N1=200),
    dict(T=300, E=5, k=2, D=200, N1=264),
    dict(T=130, E=1, k=1, D=128, N1=128),
    dict(T=700, E=3, k=1, D=136, N1=520),
    dict(T=64, E=64, k=8, D=512, N1=256),
    dict(T=900, E=4, k=2, D=264, N1=264),
    dict(T=257, E=1, k=1, D=72, N1=136),
    dict(T=900, E=4, k=2, D=320, N1=192),
    dict(T=70, E=5, k=2, D=192, N1=320),
    dict(T=300, E=2, k=2, D=640, N1=64),
    dict(T=40, E=4, k=1, D=8, N1=8),
    dict(T=300, E=2, k=1, D=16, N1=8),
    dict(T=200, E=1, k=1, D=24, N1=1000),
    dict(T=300, E=2, k=1, D=1032, N1=64),
    dict(T=600, E=200, k=5, D=64, N1=128),
]
_name = lambda c: "T{T}E{E}k{k}D{D}N{N1}".format(**c)  # noqa: E731


def _check_mlp(s, act, grad, **more):
    host = {n: f64(v) for n, v in s.items()}
    host["ids"] = s["ids"].numpy()
    m = layer(s, act, **more)
    if not grad:
        Y, bound = ref.mlp(host["X"], host["W1t"], host["W2t"], host["ids"], host["weights"], act)
        assert_within(run_mlp(m, s), Y, bound, "Y")
        return
    want = ref.mlp_grad(host["X"], host["W1t"], host["W2t"], host["ids"], host["weights"], host["dY"], act)
    got = run_mlp_grad(m, s)
    for name, (value, bound) in want.items():
        assert_within(got[name], value, bound, name)


@pytest.mark.parametrize("c", MLPS, ids=_name)
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("grad", [False, True])
def test_mlp(c, act, grad):
    _check_mlp(mlp_inputs(act=act, seed=7, **c), act, grad)


@pytest.mark.parametrize("D,N1", [(64, 256), (256, 64), (72, 264), (520, 40), (128, 64), (8, 8)])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_mlp_grad_of_narrow_matrices(D, N1, act):
    """One weight gradient has fewer rows than a CTA's tile, the other may have more."""
    _check_mlp(mlp_inputs(act=act, seed=11, T=150, D=D, N1=N1, E=3, k=2), act, True)


@pytest.mark.parametrize("k", [1, 2, 3, 5, 16, 17, 32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_choices_stored_together(k, score, renorm):
    """Tokens that share a warp's store, with logits so low that only their logarithms are safe."""
    T, E = 5003, 40
    rng = np.random.default_rng(k)
    logits = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32))
    logits[::3] -= 80.0
    logits[5::7, 2:] = -float("inf")
    c = dict(T=T, E=E, k=k, score=score, renorm=renorm, scale=1.5)
    want_ids, want_w = _oracle_route(c, logits, None)
    ids, w = _run_route(c, logits, None, True)
    assert np.array_equal(ids, want_ids)
    assert np.all(np.abs(w - want_w) <= ROUTE_TOL * np.abs(want_w) + 1e-37)


@pytest.mark.parametrize("T", [3, 90])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("how", ["dropped", "twice", "none", "one"])
def test_mlp_ids(T, act, grad, how):
    """Assignments to no expert, the same expert twice, tokens without any, one expert for all."""
    E, k = 6, 3
    rng = np.random.default_rng(T)
    ids = rng.integers(0, E - 1, (T, k)).astype(np.int32)  # the last expert gets none
    if how == "dropped":
        ids[rng.random((T, k)) < 0.4] = -1
        ids[0], ids[-1, 0] = -1, E
    elif how == "twice":
        ids[:, 1] = ids[:, 0]
    elif how == "none":
        ids[:] = -1
    else:
        ids[:] = 2
    _check_mlp(mlp_inputs(T, E, k, 96, 80, act, seed=1, ids=torch.from_numpy(ids)), act, grad)


# ------------------------------------------------------------------ use

def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("T", [5, 60, 700])
def test_layer_forward_and_backward(T):
    """The calls of a training step in a row: route, mlp, their gradients, on one stream of the
    caller's; the oracle takes the router's own choice."""
    E, k, D, N1, act = 8, 2, 136, 72, "swiglu"
    s = mlp_inputs(T, E, k, D, N1, act, seed=4)
    logits, bias = torch.randn(T, E), 0.1 * torch.randn(E)
    m = layer(s, act, score="sigmoid", renorm=True, scale=2.0)
    d = {n: v.cuda() for n, v in s.items()}
    lo, bi = logits.cuda(), bias.cuda()
    ids, w = torch.empty_like(d["ids"]), torch.empty_like(d["weights"])
    work = torch.full((max(m.info.work_bytes, m.info.grad_work_bytes),), 0xFF, dtype=torch.uint8, device="cuda")
    Y, dlo = torch.empty_like(d["X"]), torch.empty_like(lo)
    out = {n: torch.empty_like(d[n[1:]]) for n in ("dX", "dW1t", "dW2t", "dweights")}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    m.run(d["X"], lo, bi, d["W1t"], d["W2t"], ids, w, work, Y, stream=st)
    m.run_grad(d["X"], lo, d["W1t"], d["W2t"], ids, w, d["dY"], work, out["dX"], out["dW1t"], out["dW2t"],
               out["dweights"], dlo, stream=st)
    st.synchronize()
    assert m.check(work, stream=st) == (cs.OK, 0)
    host = {n: f64(v) for n, v in s.items()}
    want_ids, want_w = ref.route(f64(logits), f64(bias), k, "sigmoid", renorm=True, scale=2.0)
    got_ids, got_w = ids.cpu().numpy(), f64(w)
    assert np.array_equal(got_ids, want_ids) and np.allclose(got_w, want_w, rtol=ROUTE_TOL)
    y, bound = ref.mlp(host["X"], host["W1t"], host["W2t"], got_ids, got_w, act)
    assert_within(Y, y, bound, "Y")
    want = ref.mlp_grad(host["X"], host["W1t"], host["W2t"], got_ids, got_w, host["dY"], act)
    for name, (value, bound) in want.items():
        assert_within(out[name], value, bound, name)
    dw = f64(out["dweights"])
    want = ref.route_grad(f64(logits), got_ids, dw, "sigmoid", True, 2.0)
    q = np.abs(got_w) / 2.0  # the chosen scores over their sum
    size = 2.0 * np.abs(dw).max(axis=1, keepdims=True) * q.max(axis=1, keepdims=True)
    assert np.all(np.abs(f64(dlo) - want) <= 2 * ROUTE_TOL * size)


@pytest.mark.parametrize("T", [2, 100, 900])
def test_same_bytes_every_time_and_from_a_graph(T):
    """Repeated calls, calls with few SMs, and replays of a captured graph write the same bytes."""
    s = mlp_inputs(T, 4, 2, 192, 128, "swiglu", seed=2)
    d = {n: v.cuda() for n, v in s.items()}
    m = layer(s, "swiglu")
    work = torch.empty(max(m.info.work_bytes, m.info.grad_work_bytes), dtype=torch.uint8, device="cuda")
    Y = torch.empty_like(d["X"])
    out = [torch.empty_like(d[n]) for n in ("X", "W1t", "W2t", "weights")]

    def step(layer_, w):
        layer_.mlp(d["X"], d["W1t"], d["W2t"], d["ids"], d["weights"], w, Y)
        layer_.mlp_grad(d["X"], d["W1t"], d["W2t"], d["ids"], d["weights"], d["dY"], w, *out)

    def result():
        torch.cuda.synchronize()
        r = [_bytes(t) for t in [Y] + out]
        for t in [Y] + out:
            t.fill_(float("nan"))
        return r

    step(m, work)
    first = result()
    for other in (m, layer(s, "swiglu", num_sms=2), layer(s, "swiglu", num_sms=1)):
        step(other, work)
        # one SM takes single CTAs where more would take pairs: other widths, the same sums
        assert all(np.array_equal(a, b) for a, b in zip(first, result()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(m, work)
    for _ in range(3):
        work.fill_(0xFF)
        graph.replay()
        assert all(np.array_equal(a, b) for a, b in zip(first, result()))


def test_calls_side_by_side():
    """Two streams, each with buffers of its own."""
    cases = []
    for seed, T in ((0, 400), (1, 37)):
        s = mlp_inputs(T, 5, 2, 200, 96, "gelu", seed=seed)
        m = layer(s, "gelu")
        d = {n: v.cuda() for n, v in s.items()}
        cases.append((m, d, torch.empty(m.info.work_bytes, dtype=torch.uint8, device="cuda"), torch.empty_like(d["X"]),
                      _bytes(run_mlp(m, s)), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for m, d, work, Y, _, st in cases:
            m.mlp(d["X"], d["W1t"], d["W2t"], d["ids"], d["weights"], work, Y, stream=st)
    torch.cuda.synchronize()
    for m, d, work, Y, want, st in cases:
        assert np.array_equal(_bytes(Y), want) and m.check(work, stream=st)[0] == cs.OK


def test_routes_from_a_graph():
    c = dict(T=300, E=64, k=6, score="sigmoid", groups=8, group_limit=4, group_top=2, bias=True, renorm=True)
    logits, bias = _route_case(c, True, "none")
    m, lo, bi = _layer(c, True), logits.cuda(), bias.cuda()
    ids = torch.empty((300, 6), dtype=torch.int32, device="cuda")
    w, dl = torch.empty((300, 6), device="cuda"), torch.empty_like(lo)
    plan = torch.empty(m.info.plan_bytes // 4, dtype=torch.int32, device="cuda")

    def step():
        m.route(lo, bi, ids, w)
        m.plan(ids, plan)
        m.route_grad(lo, ids, w, dl)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lo.mul_(-1.0)  # replays read the tensors anew
    graph.replay()
    want = _oracle_route(c, -logits, bias)
    assert np.array_equal(ids.cpu().numpy(), want[0])
    assert np.array_equal(m.plan_views(plan)["slot_of"].cpu().numpy(), ref.plan(want[0], 64)["slot_of"])


# ------------------------------------------------------------------ values that do not mix

@pytest.mark.parametrize("T", [12, 200, 600])
def test_a_token_of_nans_stays_alone(T):
    s = mlp_inputs(T, 2, 1, 128, 64, "swiglu", seed=6)
    s["weights"][:] = 1.0
    clean = run_mlp(layer(s, "swiglu"), s)
    s["X"][5] = float("nan")
    s["X"][7] = float("inf")
    Y = run_mlp(layer(s, "swiglu"), s)
    assert bool(Y[5].isnan().all()) and not bool(Y[7].isfinite().all())
    keep = [t for t in range(T) if t not in (5, 7)]
    # the rows that share a scale with the two may be rounded to another fp16 (2^-11 each time),
    # and from there to another bf16
    assert bool(torch.isfinite(Y[keep]).all())
    diff = (Y[keep].float() - clean[keep].float()).abs()
    assert bool((diff <= 2.0 ** -7 * clean[keep].float().abs() + 2.0 ** -10 * clean.float().abs().max()).all())


@pytest.mark.parametrize("T", [300, 900])
def test_an_expert_of_nans_stays_alone(T):
    s = mlp_inputs(T, 4, 2, 128, 64, "swiglu", seed=8)
    m = layer(s, "swiglu")
    clean_y, clean = run_mlp(m, s), run_mlp_grad(m, s)
    s["W1t"][1], s["W2t"][1] = float("nan"), float("inf")
    Y, out = run_mlp(m, s), run_mlp_grad(m, s)
    free = (s["ids"] != 1).all(dim=1)
    assert bool(free.any()) and bool((~free).any())
    assert torch.equal(Y.cpu()[free], clean_y.cpu()[free]) and torch.equal(out["dX"].cpu()[free], clean["dX"].cpu()[free])
    for e in (0, 2, 3):
        assert torch.equal(out["dW1t"][e], clean["dW1t"][e]) and torch.equal(out["dW2t"][e], clean["dW2t"][e])
    assert torch.equal(out["dweights"].cpu()[s["ids"] != 1], clean["dweights"].cpu()[s["ids"] != 1])


def test_scaled_rows_keep_their_range():
    """Outputs far apart in size, in one tile: each token's own precision."""
    s = mlp_inputs(600, 2, 1, 128, 64, "swiglu", seed=9)
    s["X"][::2] *= 2.0 ** -9  # SwiGLU squares it: 2^-18 beside 1
    _check_mlp(s, "swiglu", False)
    s["W2t"] *= 2.0 ** 60     # beyond what fp16 holds
    _check_mlp(s, "swiglu", False)
    s["W2t"] *= 2.0 ** -120
    _check_mlp(s, "swiglu", False)


def test_offsets_beyond_32_bits():
    """Over 2^31 elements of rows by slot; the last tokens against the oracle."""
    T, E, k, D, N1 = 140000, 8, 8, 2048, 64
    ids = torch.arange(T * k, dtype=torch.int32).view(T, k) % E
    s = mlp_inputs(T, E, k, D, N1, "gelu", seed=3, ids=ids)
    m = layer(s, "gelu")
    assert m.info.slots * D > 2 ** 31
    Y = run_mlp(m, s)
    last = slice(T - 40, T)
    host = {n: f64(s[n][last] if n in ("X", "weights") else s[n]) for n in ("X", "W1t", "W2t", "weights")}
    y, bound = ref.mlp(host["X"], host["W1t"], host["W2t"], ids[last].numpy(), host["weights"], "gelu")
    assert_within(Y[last], y, bound, "Y")
    first = f64(Y[:40])
    assert np.all(np.isfinite(first))


def test_no_tokens():
    s = mlp_inputs(4, 3, 2, 64, 64, "gelu")
    for n in ("X", "dY", "ids", "weights"):
        s[n] = s[n][:0]
    m = layer(s, "gelu")
    out = run_mlp_grad_empty(m, s)
    assert all(bool((out[n] == 0).all()) for n in ("dW1t", "dW2t"))
    plan = torch.full((m.info.plan_bytes // 4,), 7, dtype=torch.int32, device="cuda")
    m.plan(s["ids"].cuda(), plan)
    assert bool((m.plan_views(plan)["counts"] == 0).all()) and bool((m.plan_views(plan)["offsets"] == 0).all())


def run_mlp_grad_empty(m, s):
    d = {n: v.cuda() for n, v in s.items()}
    out = {n: torch.full_like(d[n[1:]], float("nan")) for n in ("dX", "dW1t", "dW2t", "dweights")}
    work = torch.empty(max(16, m.info.grad_work_bytes), dtype=torch.uint8, device="cuda")
    m.mlp_grad(d["X"], d["W1t"], d["W2t"], d["ids"], d["weights"], d["dY"], work, out["dX"], out["dW1t"], out["dW2t"],
               out["dweights"])
    m.mlp(d["X"], d["W1t"], d["W2t"], d["ids"], d["weights"], work, out["dX"])
    torch.cuda.synchronize()
    return out


# ------------------------------------------------------------------ routes at the edges of their range

@pytest.mark.parametrize("E,groups,group_limit", [(20, 1, 1), (64, 1, 1), (100, 1, 1), (256, 1, 1), (300, 1, 1), (64, 8, 3),
                                                  (256, 8, 4), (160, 8, 3), (32, 4, 2), (512, 4, 2)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("forced", ["one", "top_k", "many"])
def test_route_with_biases_of_infinity(E, groups, group_limit, group_top, score, forced):
    """A bias of +inf forces its expert, one of -inf or NaN switches it off; the logits are masked too, so that
    groups hold a forced expert and nothing else."""
    T = 40
    k = min(4, group_limit * E // groups)
    rng = np.random.default_rng(E + groups + group_top)
    logits = torch.from_numpy(rng.normal(0, 1.5, (T, E)).astype(np.float32))
    logits[::2][torch.from_numpy(rng.random((T // 2, E)) < 0.9)] = float("-inf")
    bias = rng.normal(0, 0.1, E).astype(np.float32)
    off = rng.permutation(E)
    bias[off[-2]], bias[off[-1]] = -np.inf, np.nan
    bias[off[:{"one": 1, "top_k": k, "many": min(40, E - 2)}[forced]]] = np.inf
    c = dict(T=T, E=E, k=k, score=score, groups=groups, group_limit=group_limit, group_top=group_top, renorm=True)
    for top_k in {1, k}:
        c["k"] = top_k
        with np.errstate(invalid="ignore"):
            want_ids, want_w = _oracle_route(c, logits, torch.from_numpy(bias))
        ids, w = _run_route(c, logits, torch.from_numpy(bias), True)
        assert np.array_equal(ids, want_ids)
        assert np.all(np.abs(w - want_w) <= ROUTE_TOL * np.abs(want_w) + 1e-37)


# ------------------------------------------------------------------ tokens that share an expert's rows

# by the tile: gathered rows, copied rows on single CTAs, pairs of CTAs
SHARED = [dict(T=48, E=4, k=1, D=64, N1=64), dict(T=200, E=2, k=1, D=136, N1=72), dict(T=600, E=2, k=1, D=128, N1=64),
          dict(T=500, E=2, k=2, D=328, N1=192)]


@pytest.mark.parametrize("c", SHARED, ids=_name)
@pytest.mark.parametrize("down", [30, 36, 45])
@pytest.mark.parametrize("grad", [False, True])
def test_small_tokens_beside_large_ones(c, down, grad):
    """Every second token 2^-down of its neighbours: its outputs and gradients keep the precision
    that they would have alone (the oracle's bound goes by each token's own values)."""
    s = mlp_inputs(act="gelu", seed=21, **c)
    s["X"][::2] *= 2.0 ** -down
    if grad:
        s["dY"][1::2] *= 2.0 ** -down
    _check_mlp(s, "gelu", grad)


@pytest.mark.parametrize("c", SHARED, ids=_name)
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_a_huge_token_changes_no_other(c, act):
    """A finite token of 2^50 times the others' size: every other token's bytes stay as they are."""
    s = mlp_inputs(act=act, seed=22, **c)
    m = layer(s, act)
    keep = torch.arange(c["T"]) != 5
    y, dx = run_mlp(m, s).cpu(), run_mlp_grad(m, s)["dX"].cpu()
    s["X"][5] *= 2.0 ** 50
    Y = run_mlp(m, s).cpu()
    assert torch.equal(Y[keep], y[keep]) and bool(Y[5].isfinite().all())
    s["X"][5] *= 2.0 ** -50
    s["dY"][5] *= 2.0 ** 50
    dX = run_mlp_grad(m, s)["dX"].cpu()
    assert torch.equal(dX[keep], dx[keep]) and bool(dX[5].isfinite().all())


@pytest.mark.parametrize("T", [40, 600])
@pytest.mark.parametrize("D", [1024, 4096, 16384])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_dweights_of_exact_sums(T, D, act):
    """Rows with a single one: the products' sums are exact, whatever their length.  What is left:
    the sigmoid, its exponential and its division 2 steps of 2^-23 each, and half of one for each
    addition, for its argument in GeLU (weighed by less than 0.3) and for the products with it, u
    and dH; 5 + N1 / 32 additions of positive terms: 2^-23 (4 + 0.5 * (1 + 2 + 3 + 7)) < 11 steps."""
    E, N1 = 2, 64
    s = mlp_inputs(T, E, 1, D, N1, act, seed=31)
    for n in ("W1t", "W2t"):
        s[n] = (0.5 + 0.5 * s[n].float().abs().clamp(max=1.0)).to(torch.bfloat16)
    rng = np.random.default_rng(T + D)
    for n in ("X", "dY"):
        s[n].zero_()
        s[n][torch.arange(T), torch.from_numpy(rng.integers(0, D, T))] = 1.0
    want = ref.mlp_grad(*(f64(s[n]) for n in ("X", "W1t", "W2t")), s["ids"].numpy(), f64(s["weights"]), f64(s["dY"]), act)
    got = f64(run_mlp_grad(layer(s, act), s)["dweights"])
    value = want["dweights"][0]
    assert np.all(np.abs(got - value) <= 11 * 2.0 ** -23 * value)


@pytest.mark.parametrize("c", ROUTES, ids=lambda c: f"T{c['T']}E{c['E']}k{c['k']}{c['score']}")
@pytest.mark.parametrize("f32", [True, False])
def test_route_with_logits_of_infinity(c, f32):
    """Rows with one +inf, several, nothing else, and none; their weights and gradients."""
    logits, bias = _route_case(c, f32, "none", seed=3)
    rng = np.random.default_rng(c["E"])
    T, E = logits.shape
    logits[::4, rng.integers(0, E)] = float("inf")
    logits[1::4][torch.from_numpy(rng.random(logits[1::4].shape) < 0.2)] = float("inf")
    logits[1::4][torch.from_numpy(rng.random(logits[1::4].shape) < 0.2)] = float("-inf")
    logits[2::8] = float("inf")
    want_ids, want_w = _oracle_route(c, logits, bias)
    ids, w = _run_route(c, logits, bias, f32)
    assert np.array_equal(ids, want_ids)
    assert np.all(np.abs(w - want_w) <= ROUTE_TOL * np.abs(want_w) + 1e-37)
    dw = rng.normal(size=ids.shape).astype(np.float32)
    dl = torch.full_like(logits, 77).cuda()
    _layer(c, f32).route_grad(logits.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), dl)
    renorm, scale = c.get("renorm", False), c.get("scale", 1.0)
    want = ref.route_grad(f64(logits), ids, dw.astype(np.float64), c["score"], renorm, scale)
    # as in test_route_grad, the scores of at most 1 left out
    size = scale * np.abs(dw).max(axis=1, keepdims=True)
    half = 0.0 if f32 else ref.BF16
    assert np.all(np.abs(f64(dl) - want) <= 2 * ROUTE_TOL * size + half * np.abs(want))


def _grids(step):
    """The grid sizes of the kernels that step() launches."""
    class Params(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
        _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                    ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                    ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]
    cuda = ctypes.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        step()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cuda.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cuda.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        p = Params()
        assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        out.append(p.grid[0] * p.grid[1] * p.grid[2])
    return out


def test_routes_on_few_sms():
    """num_sms bounds the router's persistent kernel too; it chooses the same."""
    T, E, k = 9000, 256, 8
    logits = torch.randn(T, E, device="cuda")
    found = {}
    for sms in (0, 3, 1):
        m = cs.Moe(cs.make_moe_desc(T=T, experts=E, top_k=k, score="sigmoid", num_sms=sms))
        ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
        m.route(logits, None, ids, w)
        found[sms] = ids, w, _grids(lambda: m.route(logits, None, ids, w))
    most = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = found[0][2][0] // most  # of the persistent kernel on an SM
    assert blocks >= 1
    for sms in (3, 1):
        assert found[sms][2] == [sms * blocks]
        assert torch.equal(found[sms][0], found[0][0]) and torch.equal(found[sms][1], found[0][1])


def test_a_first_call_of_any_kind_is_enough_before_a_capture():
    """In a process of its own: one plan, then every other call for the first time inside a capture."""
    code = """
import torch, tile_level_sync_gb300 as cs
T, E, k, D, N1 = 300, 8, 2, 128, 64
bf = torch.bfloat16
def new(*s, dt=bf): return torch.randn(s, device="cuda").to(dt)
first = True
for f32 in (True, False):
    m = cs.Moe(cs.make_moe_desc(T=T, D=D, N1=N1, experts=E, top_k=k, logits_f32=f32))
    X, dY, W1, W2 = new(T, D), new(T, D), new(E, 2 * N1, D), new(E, D, N1)
    lo = new(T, E, dt=torch.float32 if f32 else bf)
    ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.ones(T, k, device="cuda")
    work = torch.empty(max(m.info.work_bytes, m.info.grad_work_bytes), dtype=torch.uint8, device="cuda")
    plan = torch.empty(m.info.plan_bytes // 4, dtype=torch.int32, device="cuda")
    out = [torch.empty_like(t) for t in (X, X, W1, W2, w, lo)]
    if first: m.plan(ids, plan)
    first = False
    def step():
        m.run(X, lo, None, W1, W2, ids, w, work, out[0])
        m.run_grad(X, lo, W1, W2, ids, w, dY, work, *out[1:])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in [ids, w] + out]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, [ids, w] + out))
print("same bytes")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "same bytes" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("grad", [False, True])
def test_no_tokens_leave_no_error(grad):
    """A call without tokens clears the error word of its buffer as any other does."""
    m = cs.Moe(cs.make_moe_desc(T=0, D=64, N1=64, experts=3, top_k=2))
    work = torch.full((max(m.info.work_bytes, m.info.grad_work_bytes),), 0xFF, dtype=torch.uint8, device="cuda")
    W1t, W2t = torch.empty(3, 128, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 64, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ids, w = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    if grad:
        m.mlp_grad(none, W1t, W2t, ids, w, none, work, none, torch.empty_like(W1t), torch.empty_like(W2t), w)
    else:
        m.mlp(none, W1t, W2t, ids, w, work, none)
    assert m.check(work) == (cs.OK, 0)


def test_check_is_refused_in_a_capture():
    """It waits for the stream: a refusal leaves the capture as it was."""
    s = mlp_inputs(60, 3, 2, 64, 64, "swiglu", seed=2)
    d = {n: v.cuda() for n, v in s.items()}
    m = layer(s, "swiglu")
    want = run_mlp(m, s)
    work, Y = torch.empty(m.info.work_bytes, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mlp(d["X"], d["W1t"], d["W2t"], d["ids"], d["weights"], work, Y)
        with pytest.raises(cs.CusyncError) as e:
            m.check(work)
    assert e.value.status == cs.ERR_UNSUPPORTED
    graph.replay()
    assert m.check(work) == (cs.OK, 0) and torch.equal(Y, want)


@pytest.mark.parametrize("T", [40, 600])
def test_gelu_gradient_far_out(T):
    """Pre-activations whose squares 32 bits do not hold: the slope there is 0 or 1."""
    s = mlp_inputs(T, 2, 1, 64, 64, "gelu", seed=41)
    s["X"][3] *= 2.0 ** 70
    out = run_mlp_grad(layer(s, "gelu"), s)
    assert all(bool(t.isfinite().all()) for t in out.values())
    e = int(s["ids"][3, 0])
    x, y, a, b = f64(s["X"][3]), f64(s["dY"][3]), f64(s["W1t"][e]), f64(s["W2t"][e])
    z, w = a @ x, float(s["weights"][3, 0])
    dz = np.where(z > 0, w * (y @ b), 0.0)
    # dZ and dX rounded to bf16, dX to fp16 between (half a step of its largest neighbour), sums of 64
    bound = 2 * ref.BF16 * (np.abs(dz) @ np.abs(a)) + ref.HALF * np.abs(dz @ a).max() + ref.BF16 * np.abs(dz @ a)
    assert np.all(np.abs(f64(out["dX"][3]) - dz @ a) <= bound)


# ------------------------------------------------------------------ long sums, borders, captures

@pytest.mark.parametrize("c", [dict(T=300, E=2, k=1, D=2056, N1=64), dict(T=70, E=4, k=2, D=1600, N1=840),
                               dict(T=400, E=3, k=2, D=1536, N1=1536)], ids=_name)
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("grad", [False, True])
def test_long_sums(c, act, grad):
    """Widths from which tiles are claimed only one ahead, in every product."""
    _check_mlp(mlp_inputs(act=act, seed=51, **c), act, grad)


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("T,E,k", [(4, 16, 8), (32, 3, 1), (16, 2, 2), (20, 40, 8), (16, 1, 1), (48, 3, 1), (127, 1, 1), (128, 1, 1)])
def test_one_token_more(T, E, k, act):
    """The same tokens on both sides of a border between kernels (32 assignments; 16 and 128 an
    expert): each within its bound, and so at most two bounds apart."""
    s = mlp_inputs(T + 1, E, k, 264, 136, act, seed=52)
    host = {n: f64(v) for n, v in s.items()}
    y, bound = ref.mlp(host["X"], host["W1t"], host["W2t"], s["ids"].numpy(), host["weights"], act)
    more = run_mlp(layer(s, act), s)
    assert_within(more, y, bound, "one token more")
    for n in ("X", "ids", "weights"):
        s[n] = s[n][:T].contiguous()
    assert_within(run_mlp(layer(s, act), s), y[:T], bound[:T], "without it")


@pytest.mark.parametrize("T", [3, 60, 700])
def test_captured_behind_other_work(T):
    """Calls captured behind a memset, a copy and another stream's kernels, which write what they read."""
    s = mlp_inputs(T, 4, 2, 128, 64, "swiglu", seed=53)
    d = {n: v.cuda() for n, v in s.items()}
    m = layer(s, "swiglu")
    want, grads = run_mlp(m, s), run_mlp_grad(m, s)
    X, dY, ids, w = (torch.full_like(d[n], 0) for n in ("X", "dY", "ids", "weights"))
    work = torch.empty(max(m.info.work_bytes, m.info.grad_work_bytes), dtype=torch.uint8, device="cuda")
    Y, out = torch.empty_like(X), {n: torch.empty_like(grads[n]) for n in ("dX", "dW1t", "dW2t", "dweights")}
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def step():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            X.copy_(d["X"])
            w.copy_(d["weights"] * 1.0)
        ids.copy_(d["ids"])
        work.zero_()
        torch.cuda.current_stream().wait_stream(side)
        m.mlp(X, d["W1t"], d["W2t"], ids, w, work, Y)
        dY.copy_(d["dY"])
        m.mlp_grad(X, d["W1t"], d["W2t"], ids, w, dY, work, *out.values())
        X.zero_()

    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in [X, dY, w, Y, *out.values()]:
            t.fill_(float("nan"))
        ids.fill_(-1)
        work.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want) and all(torch.equal(out[n], grads[n]) for n in out)


def test_gradient_offsets_beyond_32_bits():
    """Over 2^31 elements of rows by slot; the last tokens' gradients against the oracle."""
    T, E, k, D, N1 = 140000, 8, 8, 2048, 64
    ids = torch.arange(T * k, dtype=torch.int32).view(T, k) % E
    s = mlp_inputs(T, E, k, D, N1, "gelu", seed=3, ids=ids)
    m = layer(s, "gelu")
    assert m.info.slots * D > 2 ** 31
    out = run_mlp_grad(m, s)
    last = slice(T - 40, T)
    host = {n: f64(s[n][last] if n in ("X", "weights", "dY") else s[n]) for n in ("X", "W1t", "W2t", "weights", "dY")}
    want = ref.mlp_grad(host["X"], host["W1t"], host["W2t"], ids[last].numpy(), host["weights"], host["dY"], "gelu")
    for name in ("dX", "dweights"):
        assert_within(out[name][last], *want[name], name)
    assert all(bool(out[n].isfinite().all()) for n in ("dX", "dW1t", "dW2t", "dweights"))
