"""CPU tests of the mixture-of-experts layer: the oracle's pins, buffer sizes, refusals and the
binding."""

import os
import re

import numpy as np
import pytest
import torch

import tile_level_sync_gb300 as cs
from oracle import moe as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ the oracle

def test_oracle_route_by_hand():
    logits = np.log(np.array([[4.0, 2.0, 1.0, 1.0], [1.0, 1.0, 1.0, 1.0]]))
    ids, w = ref.route(logits, None, 2)
    assert ids.tolist() == [[0, 1], [0, 1]]          # equal scores: the lowest index
    assert np.allclose(w, [[0.5, 0.25], [0.25, 0.25]])
    _, w = ref.route(logits, None, 2, renorm=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0], [1.5, 1.5]])
    # a bias selects but does not weigh
    ids, w = ref.route(logits[:1], np.array([0.0, 0.0, 0.0, 9.0]), 2)
    assert ids.tolist() == [[3, 0]] and np.allclose(w, [[0.125, 0.5]])
    # two groups, one kept: by the largest key {2}, by the two largest {0}
    logits = np.log(np.array([[3.0, 3.0, 4.0, 0.5]]))
    assert ref.route(logits, None, 2, groups=2, group_limit=1)[0].tolist() == [[2, 3]]
    assert ref.route(logits, None, 2, groups=2, group_limit=1, group_top=2)[0].tolist() == [[0, 1]]


def test_oracle_route_masks():
    inf = float("inf")
    ids, w = ref.route(np.array([[-inf, 0.0, np.nan], [-inf, -inf, -inf]]), None, 2, renorm=True)
    assert ids.tolist() == [[1, -1], [-1, -1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]
    # sigmoids that underflow keep their ratio
    _, w = ref.route(np.array([[-800.0, -800.0 - np.log(3.0)]]), None, 2, "sigmoid", renorm=True)
    assert np.allclose(w, [[0.75, 0.25]])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_oracle_route_grad_is_the_difference_quotient(kind, renorm):
    rng = np.random.default_rng(0)
    l = rng.normal(size=(3, 7))
    ids = np.array([[0, 3], [6, 1], [2, -1]])
    dw = rng.normal(size=(3, 2))
    got, h = ref.route_grad(l, ids, dw, kind, renorm, 1.5), 1e-6
    for e in range(7):
        up, down = l.copy(), l.copy()
        up[:, e] += h
        down[:, e] -= h
        f = [(ref.route_weights(x, ids, kind, renorm, 1.5) * dw).sum(axis=1) for x in (up, down)]
        assert np.allclose(got[:, e], (f[0] - f[1]) / (2 * h), atol=1e-8)


def test_oracle_plan_order():
    ids = np.array([[1, 0], [1, -1], [5, 1]])
    p = ref.plan(ids, 3)
    assert p["counts"].tolist() == [1, 3, 0] and p["offsets"].tolist() == [0, 128, 256, 256]
    assert p["slot_of"].tolist() == [[128, 0], [129, -1], [-1, 130]]
    assert p["row_of"][[0, 128, 129, 130]].tolist() == [1, 0, 2, 5] and (p["row_of"] >= 0).sum() == 4
    assert len(p["row_of"]) == 512  # 6 assignments, 3 experts: 6 + 3 * 127 rows at most


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_oracle_mlp_against_loops_and_differences(act):
    T, E, k, D, N1 = 3, 2, 2, 4, 3
    rng = np.random.default_rng(1)
    G = 2 if act == "swiglu" else 1
    X, W1, W2 = rng.normal(size=(T, D)), rng.normal(size=(E, G * N1, D)), rng.normal(size=(E, D, N1))
    ids, w, dY = np.array([[0, 1], [1, 1], [-1, 0]]), rng.random((T, k)), rng.normal(size=(T, D))

    def plain(X, W1, W2, w):
        Y = np.zeros((T, D))
        for t in range(T):
            for j in range(k):
                e = ids[t, j]
                if e < 0:
                    continue
                z = W1[e] @ X[t]
                if act == "swiglu":
                    h = z[:N1] / (1 + np.exp(-z[:N1])) * z[N1:]
                else:
                    h = 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
                Y[t] += w[t, j] * (W2[e] @ h)
        return Y

    Y, bound = ref.mlp(X, W1, W2, ids, w, act)
    assert np.allclose(Y, plain(X, W1, W2, w), atol=1e-12) and np.all(bound >= 0)
    grads = ref.mlp_grad(X, W1, W2, ids, w, dY, act)
    args = {"dX": X, "dW1t": W1, "dW2t": W2, "dweights": w}
    for name, arg in args.items():
        got = grads[name][0]
        for i in np.ndindex(arg.shape):
            keep, d = arg[i], []
            for h in (1e-6, -1e-6):
                arg[i] = keep + h
                d.append((plain(X, W1, W2, w) * dY).sum())
            arg[i] = keep
            assert abs(got[i] - (d[0] - d[1]) / 2e-6) < 1e-6, (name, i)


# ------------------------------------------------------------------ sizes and refusals

GOOD = dict(T=10, D=64, N1=64, experts=8, top_k=2)


def _status(**change):
    try:
        cs.cusync_moe_info(cs.make_moe_desc(**{**GOOD, **change}))
        return cs.OK
    except cs.CusyncError as e:
        return e.status


def test_info_sizes():
    for T, E, k in ((0, 4, 2), (1, 4, 2), (100, 1, 1), (5000, 1024, 32)):
        i = cs.cusync_moe_info(cs.make_moe_desc(T=T, experts=E, top_k=k, D=64, N1=72))
        assert i.slots == ref.slots(T, E, k)
        ends = {"counts": E, "offsets": E + 1, "slot_of": T * k, "row_of": i.slots}
        at = sorted((getattr(i, n), n) for n in ends)
        for (a, n), (b, _) in zip(at, at[1:] + [(i.plan_bytes // 4, "")]):
            assert a + ends[n] <= b and a % 4 == 0
        # the rows, their hidden layer and their outputs in 16 bits at least
        assert i.work_bytes >= i.plan_bytes + i.slots * (64 + 72 + 64) * 2
        assert i.grad_work_bytes >= i.plan_bytes + i.slots * (2 * 64 + 3 * 72 + 64) * 2
    i = cs.cusync_moe_info(cs.make_moe_desc(T=10, experts=4, top_k=2))
    assert i.plan_bytes > 0 and i.work_bytes == i.grad_work_bytes == 0


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(experts=0), dict(top_k=0), dict(top_k=9), dict(groups=3), dict(groups=-1), dict(D=0), dict(N1=0),
    dict(groups=4, group_limit=5), dict(groups=4, group_limit=1, top_k=3), dict(group_top=3), dict(act=2),
    dict(score=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(num_sms=-1), dict(N1=-8)])
def test_invalid_descriptors(change):
    assert _status() == cs.OK
    assert _status(**change) == cs.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(D=60), dict(N1=60), dict(experts=1025), dict(experts=64, top_k=33), dict(experts=64, groups=64),
    dict(T=cs.MOE_MAX_ASSIGNMENTS), dict(D=1 << 21), dict(experts=1024, N1=1 << 20, D=8)])
def test_unsupported_descriptors(change):
    assert _status(**change) == cs.ERR_UNSUPPORTED


def test_largest_descriptors():
    assert _status(T=cs.MOE_MAX_ASSIGNMENTS // 2) == cs.OK
    assert _status(experts=1024, top_k=32) == cs.OK
    assert _status(experts=1024, groups=32, group_limit=1, top_k=32) == cs.OK


def test_null_and_misaligned_pointers():
    m = cs.Moe(cs.make_moe_desc(**GOOD))
    calls = {"route": 4, "route_grad": 4, "plan": 2, "mlp": 7, "mlp_grad": 11}
    for name, n in calls.items():
        for bad in range(n):
            if name == "route" and bad == 1:
                continue  # no bias is allowed
            args = [256 * (i + 1) for i in range(n)]
            for p in (None, 264):
                args[bad] = p
                with pytest.raises(cs.CusyncError) as e:
                    getattr(m, name)(*args, stream=0)
                assert e.value.status == cs.ERR_INVALID_ARG, (name, bad)
    with pytest.raises(cs.CusyncError):
        m.check(None, stream=0)


def test_tensors_are_checked():
    m = cs.Moe(cs.make_moe_desc(**GOOD))
    ids, w = torch.zeros(10, 2, dtype=torch.int32), torch.zeros(10, 2)
    logits = torch.zeros(10, 8)
    for bad, why in ((logits.double(), "float64"), (torch.zeros(10, 7), "elements"),
                     (torch.zeros(8, 10).t(), "contiguous"), (logits, "device")):
        with pytest.raises(ValueError, match=why):
            m.route(bad, None, ids, w, stream=0)
    with pytest.raises(ValueError, match="bytes"):
        m.plan(256, torch.zeros(4, dtype=torch.int32), stream=0)
    with pytest.raises(KeyError):
        cs.make_moe_desc(act="relu")


def test_nothing_to_do_needs_no_device():
    m = cs.Moe(cs.make_moe_desc(**{**GOOD, "T": 0}))
    m.route(None, None, None, None, stream=0)
    m.route_grad(None, None, None, None, stream=0)
    m.mlp(None, None, None, None, None, None, None, stream=0)


def test_binding_matches_the_header():
    src = open(os.path.join(ROOT, "include", "cusync_moe.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    found = dict(re.findall(r"\bCUSYNC_(MOE_\w+)\s*=\s*(\d+)", src) + re.findall(r"#define CUSYNC_(MOE_\w+) (\d+)", src))
    assert len(found) == 9
    for name, value in found.items():
        assert getattr(cs, name) == int(value), name
    fields = re.search(r"typedef struct \{(.*?)\} cusync_moe_desc_t;", src, re.S).group(1)
    assert re.findall(r"(\w+);", fields) == [f for f, _ in cs.cusync_moe_desc_t._fields_]
    fields = re.search(r"typedef struct \{([^}]*)\} cusync_moe_info_t;", src, re.S).group(1)
    assert re.findall(r"(\w+);", fields) == [f for f, _ in cs.cusync_moe_info_t._fields_]


# ------------------------------------------------------------------ the kernels' sources

def _sources():
    for folder in ("csrc", "csrc_moe"):
        at = os.path.join(ROOT, "tile_level_sync_gb300", folder)
        for name in sorted(os.listdir(at)):
            yield os.path.join(folder, name), open(os.path.join(at, name)).read()


def test_every_arrival_on_a_barrier_releases():
    """What a thread has read (a ring's slot, an accumulator) may be overwritten once its arrival is
    seen: only a release orders the reads before that."""
    arrivals = [(f, m.group(0)) for f, text in _sources() for m in re.finditer(r"mbarrier\.arrive[\w.:]*\.b64", text)]
    assert any(f.startswith("csrc_moe") or f.endswith("ptx.cuh") for f, _ in arrivals)
    assert [a for a in arrivals if ".release." not in a[1] and "tcgen05" not in a[1]] == []
