"""GPU parity of the norm and linear layers with the fp64 oracle (oracle/linear.py)."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tile_level_sync_gb300 as cs
from linear_helpers import (BF, F8, F32, Out, assert_checkpoint, assert_rows8, assert_within, cuda, f64, finish, layer,
                            linear_inputs, norm_inputs, oracle_grad, oracle_linear, run_linear, run_linear_grad, values)
from oracle import linear as ref
from oracle.bf16 import round_to_bf16

pytestmark = pytest.mark.gpu
EPS = 1e-5
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ norm

def _norm(M, D, kind="rms", **more):
    return cs.Norm(cs.make_norm_desc(M=M, D=D, kind=kind, eps=EPS, **more))


NORMS = [(1, 8), (3, 1000), (300, 136), (5, 2048), (2, 2056), (4, 4104), (3, 8192), (3, 8200), (2, 16392), (2, 32768), (5000, 64), (7, 256), (9, 1024), (9, 1032), (2100, 256), (2051, 1000)]


@pytest.mark.parametrize("M,D", NORMS)
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("kind", ["rms", "none"])
def test_norm(M, D, residual, kind):
    s = norm_inputs(M, D, residual)
    d = cuda(s)
    out = {"S": Out((M, D), BF), "Y": Out((M, D), BF), "Q": Out((M, D), F8), "Qs": Out((M,), F32)}
    _norm(M, D, kind).run(d["X"], d["R"], d["w"] if kind == "rms" else None, **{k: o.t for k, o in out.items()})
    S, y = ref.norm(f64(s["X"]), f64(s["R"]), f64(s["w"]), EPS, kind == "rms")
    err = ref.norm_bound(S, y, kind == "rms")
    assert_within(out["S"].t, S, 2.0 ** -8 * np.abs(S) * (1 + 2.0 ** -15), "S")
    assert_within(out["Y"].t, y, 2.0 ** -8 * np.abs(y) + 1.01 * err, "Y")
    assert_rows8(out["Q"].t, out["Qs"].t, y, err, "Q")
    assert all(o.intact() for o in out.values())


@pytest.mark.parametrize("outs", [("S",), ("Y",), ("Q", "Qs"), ("S", "Q", "Qs"), ("S", "Y")])
def test_norm_outputs_one_by_one(outs):
    M, D = 6, 520
    d = cuda(norm_inputs(M, D))
    types = {"S": ((M, D), BF), "Y": ((M, D), BF), "Q": ((M, D), F8), "Qs": ((M,), F32)}
    both = {k: Out(*types[k]) for k in types}, {k: Out(*types[k]) for k in outs}
    for o in both:
        _norm(M, D).run(d["X"], d["R"], d["w"], **{k: x.t for k, x in o.items()})
    for k in outs:
        assert torch.equal(both[0][k].buf, both[1][k].buf), k


@pytest.mark.parametrize("into", ["X", "R"])
def test_norm_adds_in_place(into):
    M, D = 9, 2600
    d = cuda(norm_inputs(M, D))
    want, Y, Z = Out((M, D), BF), Out((M, D), BF), Out((M, D), BF)
    n = _norm(M, D)
    n.run(d["X"], d["R"], d["w"], S=want.t, Y=Y.t)
    n.run(d["X"], d["R"], d["w"], S=d[into], Y=Z.t)
    assert torch.equal(d[into], want.t) and torch.equal(Y.t, Z.t)


def test_norm_of_odd_rows():
    """Zeros, the type's largest and smallest values, infinities and NaN, each in a row of its own: the rows
    between them keep their bytes."""
    M, D, inf = 12, 264, float("inf")
    s = norm_inputs(M, D, False)
    d = cuda(s)
    n = _norm(M, D)
    out = [Out((M, D), BF), Out((M, D), F8), Out((M,), F32)]
    n.run(d["X"], None, d["w"], None, *[o.t for o in out])
    before = [o.t.clone() for o in out]
    x = s["X"].clone()
    x[0] = 0
    x[2] = torch.finfo(BF).tiny
    x[4, 3], x[6, 5], x[8, 7] = inf, float("nan"), -inf
    x[10] = 2.0 ** 60
    n.run(x.cuda(), None, d["w"], None, *[o.t for o in out])
    for b, o in zip(before, out):
        assert torch.equal(*(v.view(torch.uint8).view(M, -1)[1::2] for v in (b, o.t)))
    y, q, sc = (o.t.float().cpu() for o in out)
    assert (y[0] == 0).all() and (q[0] == 0).all() and sc[0] == 2.0 ** -126
    assert torch.isfinite(y[2]).all() and torch.isfinite(q[2]).all()
    for r in (4, 8):  # squares add up to infinity: everything finite is 0 beside it
        i = (x[r].abs() == inf).nonzero().item()
        assert torch.isnan(y[r, i]) and torch.isnan(q[r, i]) and (y[r, torch.arange(D) != i] == 0).all()
        assert sc[r] == 2.0 ** -126
    assert torch.isnan(y[6]).all() and torch.isnan(q[6]).all()
    assert_within(y[10], f64(s["w"])[None].repeat(1, 0)[0], 2.0 ** -7 * np.abs(f64(s["w"])), "large")
    # the addition alone: the finite values of such rows stay, and scale the row
    m = _norm(M, D, "none")
    m.run(x.cuda(), None, None, None, None, out[1].t, out[2].t)
    q, sc = out[1].t.float().cpu(), out[2].t.cpu()
    for r in (4, 6, 8):
        ok = torch.isfinite(x[r])
        assert torch.isnan(q[r][~ok]).all() and torch.isfinite(q[r][ok]).all()
        assert abs(sc[r] - x[r][ok].float().abs().max() / 448) <= 2.0 ** -22 * sc[r]


@pytest.mark.parametrize("M,D", NORMS + [(2000, 1000), (700, 8200), (330, 16392), (330, 32768), (3000, 8), (9000, 256), (3000, 1024), (2500, 1032),
                                         (1300, 4096), (400, 12288), (400, 20480), (200, 1024)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_grad(M, D, residual):
    s = norm_inputs(M, D, residual)
    d = cuda(s)
    n = _norm(M, D)
    dX, dw, work = Out((M, D), BF), Out((D,), BF), Out((n.info.grad_work_bytes,), torch.uint8)
    n.run_grad(d["X"], d["w"], d["dY"], d["R"], work.t, dX.t, dw.t)
    want = ref.norm_grad(f64(s["X"]), f64(s["w"]), f64(s["dY"]), f64(s["R"]), EPS)
    assert_within(dX.t, *want["dX"], "dX")
    assert_within(dw.t, *want["dw"], "dw")
    assert dX.intact() and dw.intact() and work.intact()


@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 127, 2.0 ** -60])
def test_norm_of_rows_whose_squares_leave_32_bits(size):
    M, D, eps = 5, 264, 1e-6 if size > 1 else 0.0
    s = norm_inputs(M, D, False)
    g = torch.Generator().manual_seed(4)
    s["X"] = (torch.randn(M, D, generator=g).clamp(-1.9, 1.9) * size).to(BF)
    s["X"][3] = 0 if eps else 1
    d = cuda(s)
    n = cs.Norm(cs.make_norm_desc(M=M, D=D, eps=eps))
    Y, Q, Qs, dX, dw = Out((M, D), BF), Out((M, D), F8), Out((M,), F32), Out((M, D), BF), Out((D,), BF)
    n.run(d["X"], None, d["w"], Y=Y.t, Q=Q.t, Qs=Qs.t)
    S, y = ref.norm(f64(s["X"]), None, f64(s["w"]), eps)
    err = ref.norm_bound(S, y) + 2.0 ** -20 * np.abs(y)  # a factor below 2^-126 has 20 bits
    assert_within(Y.t, y, 2.0 ** -8 * np.abs(y) + 1.01 * err, "Y")
    assert_rows8(Q.t, Qs.t, y, err, "Q")
    work = torch.empty(n.info.grad_work_bytes, dtype=torch.uint8, device="cuda")
    n.run_grad(d["X"], d["w"], d["dY"], None, work, dX.t, dw.t)
    want = ref.norm_grad(f64(s["X"]), f64(s["w"]), f64(s["dY"]), None, eps)
    value, bound = want["dX"]
    assert_within(dX.t, value, bound + 2.0 ** -20 * np.abs(value).max(axis=1, keepdims=True) + 2.0 ** -133, "dX")
    value, bound = want["dw"]
    assert_within(dw.t, value, bound + 2.0 ** -18 * np.abs(f64(s["dY"])).sum(axis=0), "dw")


def _norm_and_gradient_of(M, D, X, dY, eps=0.0):
    """Y, 8-bit rows and gradients within the bounds of rows whose squares fit."""
    s = dict(norm_inputs(M, D, False), X=X, dY=dY)
    d, n = cuda(s), cs.Norm(cs.make_norm_desc(M=M, D=D, eps=eps))
    Y, Q, Qs, dX, dw = Out((M, D), BF), Out((M, D), F8), Out((M,), F32), Out((M, D), BF), Out((D,), BF)
    n.run(d["X"], None, d["w"], Y=Y.t, Q=Q.t, Qs=Qs.t)
    S, y = ref.norm(f64(s["X"]), None, f64(s["w"]), eps)
    err = ref.norm_bound(S, y)
    assert_within(Y.t, y, 2.0 ** -8 * np.abs(y) + 1.01 * err, "Y")
    assert_rows8(Q.t, Qs.t, y, err, "Q")
    work = Out((n.info.grad_work_bytes,), torch.uint8)
    n.run_grad(d["X"], d["w"], d["dY"], None, work.t, dX.t, dw.t)
    want = ref.norm_grad(f64(s["X"]), f64(s["w"]), f64(s["dY"]), None, eps)
    value, bound = want["dX"]
    assert_within(dX.t, value, bound + 2.0 ** -133, "dX")  # the type's smallest step, of which half is a rounding
    assert_within(dw.t, *want["dw"], "dw")
    assert all(o.intact() for o in (Y, Q, Qs, dX, dw, work))


ENDS = [(5, 264), (1100, 264), (5, 1024), (1100, 1024), (3, 4104), (3, 8200), (3, 32768)]


@pytest.mark.parametrize("M,D", ENDS)
def test_norm_of_rows_of_the_largest_values(M, D):
    g = torch.Generator().manual_seed(4 + M + D)
    sign = torch.randint(0, 2, (M, D), generator=g).double() * 2 - 1
    X = (sign * torch.finfo(BF).max * (1 - 2.0 ** -3 * torch.randint(0, 5, (M, D), generator=g))).to(BF)
    _norm_and_gradient_of(M, D, X, norm_inputs(M, D, False)["dY"])


@pytest.mark.parametrize("M,D", ENDS)
def test_norm_of_rows_of_the_smallest_values(M, D):
    """Whole multiples of 2^-133, whose rows' factors are beyond 32 bits, and one row with a single such value."""
    g = torch.Generator().manual_seed(4 + M + D)
    X = torch.randint(-7, 8, (M, D), generator=g).double()
    X[:, 0] = 1
    X[1, 1:] = 0
    dY = norm_inputs(M, D, False)["dY"].float() * 2.0 ** -24  # the gradients are divided by the rows' size
    _norm_and_gradient_of(M, D, (X * 2.0 ** -133).to(BF), dY.to(BF))


@pytest.mark.parametrize("M,D", [(5, 264), (1100, 264), (3, 8200), (2, 20480)])
@pytest.mark.parametrize("eps", [2.0 ** 127, 2.0 ** 110, 2.0 ** -120, 2.0 ** -140])
def test_norm_of_far_out_eps(M, D, eps):
    """eps beside rows of ordinary values, and beside rows whose squares are about as large as it is."""
    g = torch.Generator().manual_seed(6 + M + D)
    X = torch.randn(M, D, generator=g).double()
    X[1] *= 2.0 ** round(np.log2(eps) / 2)
    _norm_and_gradient_of(M, D, X.to(BF), norm_inputs(M, D, False)["dY"], eps)


@pytest.mark.parametrize("M,D", [(5, 264), (1100, 264), (3, 2056), (3, 8200), (2, 20480)])
@pytest.mark.parametrize("size,weight", [(2.0 ** 59, 2.0 ** 70), (2.0 ** -45, 2.0 ** -110), (2.0 ** 100, 2.0 ** 100),
                                         (2.0 ** -100, 2.0 ** -100), (2.0 ** 40, 2.0 ** -60)])
def test_norm_row_scales_of_far_out_weights(M, D, size, weight):
    """A row's scale is of its y, whose factors' product S w may lie outside of 32 bits where y does not."""
    s = norm_inputs(M, D, False)
    s["X"] = (torch.randn(M, D, generator=torch.Generator().manual_seed(11)) * size).to(BF)
    s["w"] = (s["w"].float() * weight).to(BF)
    d = cuda(s)
    Y, Q, Qs = Out((M, D), BF), Out((M, D), F8), Out((M,), F32)
    cs.Norm(cs.make_norm_desc(M=M, D=D, eps=0.0)).run(d["X"], None, d["w"], Y=Y.t, Q=Q.t, Qs=Qs.t)
    S, y = ref.norm(f64(s["X"]), None, f64(s["w"]), 0.0)
    err = ref.norm_bound(S, y)
    assert_within(Y.t, y, 2.0 ** -8 * np.abs(y) + 1.01 * err, "Y")
    assert_rows8(Q.t, Qs.t, y, err, "Q")


@pytest.mark.parametrize("M,D", [(5, 264), (1100, 264), (3, 8200)])
@pytest.mark.parametrize("size,weight,eps", [(2.0 ** -78, 2.0 ** -78, 2.0 ** -20), (2.0 ** -78, 2.0 ** -78, 2.0 ** -98),
                                             (2.0 ** -70, 2.0 ** -70, 2.0 ** -98), (2.0 ** -60, 2.0 ** -60, 2.0 ** -98),
                                             (2.0 ** -60, 2.0 ** -60, 2.0 ** -60)])
def test_norm_row_scales_of_products_near_zero(M, D, size, weight, eps):
    """max |S w| is 0 in 32 bits, or has few of them; max |y| / 448 is above and below the least scale."""
    s = norm_inputs(M, D, False)
    s["X"] = (torch.randn(M, D, generator=torch.Generator().manual_seed(13)) * size).to(BF)
    s["w"] = (s["w"].float() * weight).to(BF)
    s["X"][1] = 0
    d = cuda(s)
    Q, Qs = Out((M, D), F8), Out((M,), F32)
    cs.Norm(cs.make_norm_desc(M=M, D=D, eps=eps)).run(d["X"], None, d["w"], Q=Q.t, Qs=Qs.t)
    S, y = ref.norm(f64(s["X"]), None, f64(s["w"]), eps)
    assert_rows8(Q.t, Qs.t, y, ref.norm_bound(S, y) + 2.0 ** -149, "Q")  # y's own step there
    assert Qs.t[1] == 2.0 ** -126 and (Q.t[1].float() == 0).all()


@pytest.mark.parametrize("M,D", [(3, 264), (1100, 264), (3, 8200)])
@pytest.mark.parametrize("size,odd", [(1.0, 100.0), (2.0 ** -7, 0.5)])  # S w beyond 32 bits, and S w / rms alone
def test_norm_values_beyond_32_bits_do_not_count_for_a_scale(M, D, size, odd):
    s = norm_inputs(M, D, False)
    s["X"] = (torch.randn(M, D, generator=torch.Generator().manual_seed(12)) * size).to(BF)
    s["X"][:, 7], s["w"][7] = odd, torch.finfo(BF).max
    d = cuda(s)
    Y, Q, Qs = Out((M, D), BF), Out((M, D), F8), Out((M,), F32)
    _norm(M, D).run(d["X"], None, d["w"], Y=Y.t, Q=Q.t, Qs=Qs.t)
    S, y = ref.norm(f64(s["X"]), None, f64(s["w"]), EPS)
    assert (y[:, 7] > 2.0 * 2.0 ** 128).all()
    assert torch.isinf(Y.t[:, 7].float()).all() and torch.isnan(Q.t[:, 7].float()).all()
    keep = np.arange(D) != 7
    assert_rows8(Q.t.float()[:, torch.from_numpy(keep).cuda()], Qs.t, y[:, keep], ref.norm_bound(S, y)[:, keep], "Q")


def test_norm_grad_in_place_and_without_dw():
    M, D = 700, 1032
    d = cuda(norm_inputs(M, D))
    n = _norm(M, D)
    work = torch.empty(n.info.grad_work_bytes, dtype=torch.uint8, device="cuda")
    dX, dw, again = torch.empty_like(d["X"]), torch.empty_like(d["w"]), torch.empty_like(d["w"])
    n.run_grad(d["X"], d["w"], d["dY"], d["R"], work, dX, dw)
    for into in ("dY", "R"):
        t = {k: d[k].clone() for k in ("dY", "R")}
        n.run_grad(d["X"], d["w"], t["dY"], t["R"], work, t[into], again)
        assert torch.equal(t[into], dX) and torch.equal(again, dw)
    t = torch.empty_like(dX)
    n.run_grad(d["X"], d["w"], d["dY"], d["R"], work, t, None)
    assert torch.equal(t, dX)
    few = _norm(M, D, num_sms=3)
    few.run_grad(d["X"], d["w"], d["dY"], d["R"], work, t, again)
    assert torch.equal(t, dX)  # fewer blocks add dw in another order
    want = ref.norm_grad(f64(d["X"]), f64(d["w"]), f64(d["dY"]), f64(d["R"]), EPS)
    assert_within(again, *want["dw"], "dw")


def test_norm_gradient_against_differences():
    """The gradient's dot product with a direction, against the forward pass's difference along it."""
    M, D, h = 4, 256, 2.0 ** -5
    s = norm_inputs(M, D, False, seed=3)
    s["X"] = torch.randn(M, D, generator=torch.Generator().manual_seed(1)).to(BF)
    n = _norm(M, D)
    dX, dw = torch.empty(M, D, dtype=BF, device="cuda"), torch.empty(D, dtype=BF, device="cuda")
    work = torch.empty(n.info.grad_work_bytes, dtype=torch.uint8, device="cuda")
    d = cuda(s)
    n.run_grad(d["X"], d["w"], d["dY"], None, work, dX, dw)
    step = torch.sign(torch.randn(M, D, generator=torch.Generator().manual_seed(2)))
    ends = []
    for sign in (1, -1):
        x = (s["X"].float() + sign * h * step).to(BF)
        y = torch.empty(M, D, dtype=BF, device="cuda")
        n.run(x.cuda(), None, d["w"], Y=y)
        ends.append((f64(x), f64(y)))
    (xa, ya), (xb, yb) = ends
    along, seen = (f64(dX) * (xa - xb)).sum(), ((ya - yb) * f64(s["dY"])).sum()
    # y's roundings, 2^-8 each way, the gradient's, and the third derivative's h^2
    slack = 2.0 ** -8 * ((np.abs(ya) + np.abs(yb)) * np.abs(f64(s["dY"]))).sum() ** 1.0
    assert abs(along - seen) <= slack and slack < 20 * abs(h) * M * D


ROUNDINGS = 6.0  # sums of independent errors e_i exceed 6 sqrt(sum e_i^2) with a probability of 3e-8 at most (Hoeffding)


def test_norm_gradient_along_itself_and_along_the_rows():
    """The gradient's products with two directions against the forward pass's differences: its own signs, along which every
    part of it counts, and the rows S, along which y does not change and the term of the mean does all.  Wrong gradients
    have to be found out by the same bounds."""
    M, D, h, eps = 4, 256, 2.0 ** -5, 1e-5
    g = torch.Generator().manual_seed(1)
    s = norm_inputs(M, D, False, seed=3)
    s["X"] = torch.randn(M, D, generator=g).to(BF)
    s["w"] = torch.exp(torch.randn(D, generator=g)).to(BF)
    # the sign of S w in dY makes the mean of g S large
    s["dY"] = (torch.sign(s["X"].float() * s["w"].float()) * torch.randn(M, D, generator=g).abs()).to(BF)
    n = _norm(M, D)
    dX, dw = torch.empty(M, D, dtype=BF, device="cuda"), torch.empty(D, dtype=BF, device="cuda")
    work = torch.empty(n.info.grad_work_bytes, dtype=torch.uint8, device="cuda")
    d = cuda(s)
    n.run_grad(d["X"], d["w"], d["dY"], None, work, dX, dw)
    S, w, dY = f64(s["X"]), f64(s["w"]), f64(s["dY"])
    exact = ref.norm_grad(S, w, dY, None, eps)["dX"][0]
    r = 1 / np.sqrt((S * S).mean(axis=1, keepdims=True) + eps)
    wrong = {"zero": 0 * exact, "negated": -exact, "twice": 2 * exact, "without w": r * (dY - S * r * (dY * S * r).mean(axis=1, keepdims=True)),
             "without the mean": r * w * dY}
    found = set()
    for step in (np.sign(exact), S):
        ends = []
        for sign in (1, -1):
            x = torch.from_numpy(S + sign * h * step).to(BF)
            y = torch.empty(M, D, dtype=BF, device="cuda")
            n.run(x.cuda(), None, d["w"], Y=y)
            ends.append((f64(x), f64(y)))
        (xa, ya), (xb, yb) = ends
        seen = ((ya - yb) * dY).sum()
        # y's roundings, 2^-8 of the value each; the difference's own distance from the first derivative
        noise = ROUNDINGS * 2.0 ** -8 * np.sqrt((ya ** 2 * dY ** 2).sum() + (yb ** 2 * dY ** 2).sum())
        curve = abs(((ref.norm(xa, None, w, eps)[1] - ref.norm(xb, None, w, eps)[1]) * dY).sum() - (exact * (xa - xb)).sum())
        own = ROUNDINGS * 2.0 ** -8 * np.sqrt((exact ** 2 * (xa - xb) ** 2).sum())  # dX's roundings
        assert abs((f64(dX) * (xa - xb)).sum() - seen) <= noise + curve + own
        found |= {k for k, v in wrong.items() if abs((v * (xa - xb)).sum() - seen) > noise + curve + own}
    assert found == set(wrong)


# ------------------------------------------------------------------ linear: forward

# few tiles (clusters that divide the reduction), then many (pairs); ragged in every dimension
SMALL = [(1, 64, 128), (1, 1000, 776), (2, 8, 8), (16, 4096, 264), (17, 136, 200), (33, 520, 328), (64, 2048, 1024),
         (100, 1000, 776), (129, 256, 128), (333, 1000, 776)]
PAIRS = [(1030, 72, 2312), (2048, 256, 1536), (1281, 520, 2056), (48, 384, 6992), (129, 384, 6992), (20000, 64, 8), (20000, 16, 40),
         (300, 64, 20008)]


@pytest.mark.parametrize("M,K,N", SMALL + PAIRS)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_linear(M, K, N, act, dtype):
    if dtype == "e4m3":
        K = -(-K // 16) * 16
    s = linear_inputs(M, K, N, act, dtype)
    m = layer(M, K, N, act, dtype)
    got = run_linear(m, s, checkpoint=True)
    Y, bound, z, dz = oracle_linear(s, act)
    assert_within(got["Y"], Y, bound, "Y")
    assert_checkpoint(got["Zq"], got["Ze"], z, dz, m.info.parts, "Z")
    # without the checkpoint, the same Y
    assert torch.equal(run_linear(m, s)["Y"], got["Y"])


@pytest.mark.parametrize("M,K,N", [(33, 16384, 136), (1, 16400, 1032), (600, 16400, 2056)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_linear_long_sums(M, K, N, dtype):
    """Sums of whole numbers that 24 bits hold come out exactly, whatever the order; others within the bound."""
    g = torch.Generator().manual_seed(M)
    s = linear_inputs(M, K, N, "none", dtype, bias=False, residual=False)
    m = layer(M, K, N, "none", dtype)
    Y, bound, _, _ = oracle_linear(s, "none")
    assert_within(run_linear(m, s)["Y"], Y, bound, "Y")
    x, w = torch.randint(-8, 9, (M, K), generator=g).float(), torch.randint(-8, 9, (N, K), generator=g).float()
    w[:, 128:] *= torch.rand(N, 1, generator=g) < 0.5
    s["X"], s["Wt"] = (t.to(F8 if dtype == "e4m3" else BF) for t in (x, w))
    if dtype == "e4m3":
        s["Xs"], s["Ws"] = torch.ones(M), torch.full((N,), 2.0 ** -4)
        w = w * 2.0 ** -4
    want = (x.double() @ w.double().t()).numpy()
    assert np.array_equal(f64(run_linear(m, s)["Y"]), round_to_bf16(want))


@pytest.mark.parametrize("M,K,N", [(5, 1000, 776), (1281, 520, 2056)])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_linear_without_bias_or_residual(M, K, N, bias, residual, act):
    s = linear_inputs(M, K, N, act, bias=bias, residual=residual)
    Y, bound, _, _ = oracle_linear(s, act)
    assert_within(run_linear(layer(M, K, N, act), s)["Y"], Y, bound, "Y")


@pytest.mark.parametrize("M,K,N", [(5, 1000, 776), (1281, 520, 2056)])
def test_linear_adds_to_its_residual_in_place(M, K, N):
    s = linear_inputs(M, K, N, "relu")
    m = layer(M, K, N, "relu")
    want = run_linear(m, s)["Y"]
    d = cuda(s)
    m.run(d["X"], d["Wt"], torch.empty(m.info.work_bytes, dtype=torch.uint8, device="cuda"), d["R"], bias=d["bias"], R=d["R"])
    assert torch.equal(d["R"], want)


@pytest.mark.parametrize("num_sms", [1, 2, 7])
@pytest.mark.parametrize("M,K,N", [(20, 1000, 776), (1281, 520, 2056)])
def test_linear_on_few_sms(num_sms, M, K, N):
    s = linear_inputs(M, K, N, "swiglu")
    Y, bound, _, _ = oracle_linear(s, "swiglu")
    assert_within(run_linear(layer(M, K, N, "swiglu", num_sms=num_sms), s)["Y"], Y, bound, "Y")


@pytest.mark.parametrize("num_sms", [1, 2, 3])
@pytest.mark.parametrize("M,K,N", [(100, 1024, 776), (333, 1008, 776)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_linear_and_gradient_on_few_sms(num_sms, M, K, N, dtype):
    """Reductions long enough for clusters of eight, of which one SM holds none."""
    s = linear_inputs(M, K, N, "gelu", dtype)
    Y, bound, _, _ = oracle_linear(s, "gelu")
    m = layer(M, K, N, "gelu", dtype, num_sms=num_sms)
    assert_within(run_linear(m, s)["Y"], Y, bound, "Y")
    s = linear_inputs(M, K, N, "gelu", dtype, grad=True)
    got = run_linear_grad(m, s)
    for name, (value, bound) in oracle_grad(s, "gelu").items():
        assert_within(got[name], value, bound, name)


@pytest.mark.parametrize("M,K,N", [(70, 1000, 776), (1281, 520, 2056)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
def test_odd_values_stay_in_their_rows(M, K, N, act):
    """Rows of infinities, NaN and the type's largest values leave the other rows' bytes alone."""
    s = linear_inputs(M, K, N, act)
    m = layer(M, K, N, act)
    clean = run_linear(m, s, checkpoint=True)
    odd = [0, 33, M - 2]
    s["X"][0, 5], s["X"][33, 7], s["X"][M - 2] = float("inf"), float("nan"), torch.finfo(BF).max
    got = run_linear(m, s, checkpoint=True)
    keep = torch.ones(M, dtype=torch.bool)
    keep[odd] = False
    for k in clean:
        a, b = (t[k].view(M, -1).view(torch.uint8)[keep.cuda()] for t in (clean, got))
        assert torch.equal(a, b), k
    assert torch.isnan(got["Y"][33].float()).all() and torch.isnan(got["Zq"][33].float()).all()
    assert torch.isnan(got["Zq"][0].float()).all() and (got["Ze"][0] == 1).all()
    if act in ("none", "relu"):  # +-inf, times weights of either sign
        want = f64(s["Wt"])[:, 5] * np.inf
        y = f64(got["Y"][0]).reshape(-1)
        assert np.array_equal(y, np.maximum(want, 0) + f64(s["R"][0]) if act == "relu" else want)


@pytest.mark.parametrize("M,K,N", [(5, 1008, 776), (1281, 528, 2056)])
@pytest.mark.parametrize("xs,ws", [(2.0 ** 118, 1.0), (-2.0 ** 118, 1.0), (2.0 ** -118, 2.0 ** 100), (1.0, -1.0)])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_scales_far_out_and_negative(M, K, N, xs, ws, act):
    """Rows and weights whose values, and whose products' sums, bf16 holds: what lies between stays within 32 bits, too."""
    s = linear_inputs(M, K, N, act, "e4m3", bias=False, residual=False)
    s["Xs"], s["Ws"] = s["Xs"] * xs, s["Ws"] * ws
    m = layer(M, K, N, act, "e4m3")
    got = run_linear(m, s, checkpoint=True)
    Y, bound, z, dz = oracle_linear(s, act)
    assert_within(got["Y"], Y, bound, "Y")
    assert_checkpoint(got["Zq"], got["Ze"], z, dz, 1, "Z")


def test_checkpoint_of_odd_blocks():
    """Pre-activations of one large value beside small ones, and of zeros: through a bias on zero inputs."""
    M, K, N = 3, 64, 72
    s = linear_inputs(M, K, N, "none", bias=True, residual=False)
    s["X"].zero_()
    b = torch.full((N,), 2.0 ** -20)
    b[0], b[32:64] = 1e30, 0.0
    b[64:] = torch.tensor([448.0, 449.0, 2.0 ** -9, 2.0 ** -8, 3.0, -3.0, 0.1, -448.0])
    s["bias"] = b.to(BF)
    got = run_linear(layer(M, K, N, "none"), s, checkpoint=True)
    z = np.repeat(f64(s["bias"])[None], M, 0)
    q, e = ref.checkpoint(z, 1)
    assert np.array_equal(got["Ze"].cpu().numpy(), e) and np.array_equal(f64(got["Zq"]), q)


# ------------------------------------------------------------------ linear: gradients

@pytest.mark.parametrize("M,K,N", [(1, 64, 128), (3, 1000, 776), (17, 136, 200), (100, 264, 520), (333, 1000, 776),
                                   (1030, 264, 520), (700, 1544, 1032), (1300, 2056, 2056), (2050, 2048, 1024),
                                   (20000, 64, 8), (20000, 16, 40), (130, 64, 8200), (5000, 136, 72)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_linear_grad(M, K, N, act, dtype):
    if dtype == "e4m3":
        K = -(-K // 16) * 16
    s = linear_inputs(M, K, N, act, dtype, grad=True)
    got = run_linear_grad(layer(M, K, N, act, dtype), s)
    for name, (value, bound) in oracle_grad(s, act).items():
        assert_within(got[name], value, bound, name)


@pytest.mark.parametrize("M,K,N", [(17, 144, 200), (1300, 1040, 1032)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_grad_of_negative_scales(M, K, N, act):
    s = linear_inputs(M, K, N, act, "e4m3", grad=True)
    s["Xs"][1::2] *= -1
    m = layer(M, K, N, act, "e4m3")
    got = run_linear_grad(m, s)
    for name, (value, bound) in oracle_grad(s, act).items():
        assert_within(got[name], value, bound, name)
    # a row that stands for NaN: dX and dbias do not see it, dWt is NaN
    s["Xs"][2] = float("nan")
    odd = run_linear_grad(m, s)
    assert torch.isnan(odd["dWt"].float()).all()
    assert torch.equal(odd["dbias"], got["dbias"]) and torch.isfinite(odd["dX"].float()).all()


@pytest.mark.parametrize("want", [("dX",), ("dWt",), ("dbias",), ("dX", "dWt"), ("dX", "dbias")])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_linear_grad_one_by_one(want, act, dtype):
    M, K, N = 90, 208, 264
    s = linear_inputs(M, K, N, act, dtype, grad=True)
    m = layer(M, K, N, act, dtype)
    whole, some = run_linear_grad(m, s), run_linear_grad(m, s, want)
    # dX beside dWt of 8-bit rows is of operands rounded times the rows' fractions: other bytes
    same = [k for k in want if not (k == "dX" and dtype == "e4m3" and act != "none" and "dWt" not in want)]
    assert all(torch.equal(whole[k], some[k]) for k in same)
    if same != list(want):
        assert_within(some["dX"], *oracle_grad(dict(s, X=s["Wt"][:1].expand(M, K), Xs=None), act)["dX"], "dX")


def test_linear_grad_needs_only_what_it_reads():
    M, K, N = 40, 64, 72
    s = linear_inputs(M, K, N, "gelu", grad=True)
    m, d = layer(M, K, N, "gelu"), cuda(s)
    whole = run_linear_grad(m, s)
    work = torch.empty(m.info.grad_work_bytes, dtype=torch.uint8, device="cuda")
    dX, dWt, db = (torch.empty_like(whole[k]) for k in ("dX", "dWt", "dbias"))
    m.run_grad(None, d["Wt"], d["dY"], work, dX, None, Zq=d["Zq"], Ze=d["Ze"])
    m.run_grad(d["X"], None, d["dY"], work, None, dWt, Zq=d["Zq"], Ze=d["Ze"])
    m.run_grad(None, None, d["dY"], work, None, None, db, Zq=d["Zq"], Ze=d["Ze"])
    assert torch.equal(dX, whole["dX"]) and torch.equal(dWt, whole["dWt"]) and torch.equal(db, whole["dbias"])


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_slopes_far_out(act):
    """Pre-activations up to the checkpoint's largest: slopes of 0 and 1 (SwiGLU: of up), no NaN."""
    M, K, N = 8, 64, 64
    s = linear_inputs(M, K, N, act, grad=True)
    G = 2 if act == "swiglu" else 1
    z = np.zeros((M, G, N))
    z[:, 0] = np.array([1e38, -1e38, 1e20, -1e20, 300, -300, 60, -60])[:, None]
    if G == 2:
        z[:, 1] = np.where(np.abs(z[:, 0]) > 1e15, 1e-6, 2.0)
    q, e = ref.checkpoint(z.reshape(M, G * N), G)
    s["Zq"], s["Ze"] = torch.from_numpy(q).float().to(F8), torch.from_numpy(e.astype(np.uint8))
    got = run_linear_grad(layer(M, K, N, act), s)
    # SwiGLU's up gradients are dY 1e38 here, times X up to 10 and more: beyond 3.4e38 there is no finite
    # result.  Everything whose magnitudes add up to less than that is finite.
    dz, _ = ref.slope(z.reshape(M, G * N), f64(s["dY"]), act)
    most = {"dX": np.abs(dz) @ np.abs(f64(s["Wt"])), "dWt": np.abs(dz).T @ np.abs(f64(s["X"])), "dbias": np.abs(dz).sum(axis=0)}
    for k in got:
        v = f64(got[k])
        assert not np.isnan(v).any() and np.isfinite(v[most[k] < 3e38]).all(), k
    if act == "gelu":
        d = f64(s["dY"])
        d[1::2] = 0
        assert_within(got["dX"], d @ f64(s["Wt"]), 2.0 ** -7 * (np.abs(d) @ np.abs(f64(s["Wt"]))), "dX")


@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_gradient_of_preactivations_that_are_not_finite(act, dtype):
    """NaN, what a checkpoint holds of infinities and NaN, reaches the gradients that it is part of, and no other byte."""
    M, K, N = 70, 64, 72
    s = linear_inputs(M, K, N, act, dtype, grad=True)
    m = layer(M, K, N, act, dtype)
    clean = run_linear_grad(m, s)
    s["Zq"].view(torch.uint8)[33, 5] = 0x7F
    odd = run_linear_grad(m, s)
    assert torch.isnan(odd["dX"][33].float()).all() and torch.isnan(odd["dWt"][5].float()).all() and torch.isnan(odd["dbias"][5])
    rows, cols = torch.arange(M) != 33, torch.ones(m.info.parts * N, dtype=torch.bool)
    cols[5::N] = False  # SwiGLU: the up column beside the gate's
    assert torch.equal(odd["dX"][rows.cuda()], clean["dX"][rows.cuda()])
    for k in ("dWt", "dbias"):
        assert torch.equal(odd[k][cols.cuda()], clean[k][cols.cuda()]), k


def test_linear_gradient_against_differences():
    """dX along a direction, against differences of the forward pass on the device."""
    M, K, N, h = 32, 128, 192, 2.0 ** -4
    for act in ("gelu", "swiglu"):
        s = linear_inputs(M, K, N, act, residual=False, seed=5)
        m = layer(M, K, N, act)
        fwd = run_linear(m, s, checkpoint=True)
        s["Zq"], s["Ze"] = fwd["Zq"].cpu(), fwd["Ze"].cpu()
        dX = f64(run_linear_grad(m, s)["dX"])
        g = torch.Generator().manual_seed(9)
        step = torch.sign(torch.randn(M, K, generator=g))
        ends = []
        for sign in (1, -1):
            t = dict(s, X=(s["X"].float() + sign * h * step).to(BF))
            ends.append((f64(t["X"]), f64(run_linear(m, t)["Y"])))
        (xa, ya), (xb, yb) = ends
        along, seen = dX * (xa - xb), (ya - yb) * f64(s["dY"])
        # the checkpoint's 2^-4 of a slope, at random over M N terms; a missing factor or part is far above
        assert abs(along.sum() - seen.sum()) <= 0.1 * np.sqrt((seen ** 2).sum() * 9 + (along ** 2).sum() * 9), act


@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
def test_linear_gradient_along_its_parts(act):
    """dX's products with the signs of its parts (of the gate and the up projection, or the whole and what the slope takes
    away), against differences of the forward pass on the device, bounded by the roundings and by what 64 bits give for the
    checkpoint's and the difference's share.
    A gradient that lacks a part, a factor or the slope has to be found out by the same bounds."""
    M, K, N, h = 32, 128, 192, 2.0 ** -6
    s = linear_inputs(M, K, N, act, residual=False, seed=5)
    m = layer(M, K, N, act)
    fwd = run_linear(m, s, checkpoint=True)
    s["Zq"], s["Ze"] = fwd["Zq"].cpu(), fwd["Ze"].cpu()
    dX = f64(run_linear_grad(m, s)["dX"])
    X, Wt, dY, bias = f64(s["X"]), f64(s["Wt"]), f64(s["dY"]), f64(s["bias"])
    z = X @ Wt.T + bias
    dz, kept = ref.slope(z, dY, act)[0], ref.slope(values(s, m.info.parts), dY, act)[0]
    exact = dz @ Wt
    cut = [slice(0, N), slice(N, 2 * N)][:m.info.parts]
    parts = [dz[:, c] @ Wt[c] for c in cut]
    wrong = {"zero": 0 * exact, "negated": -exact, "twice": 2 * exact}
    if act == "swiglu":
        wrong.update({"without gate": parts[1], "without up": parts[0], "parts exchanged": dz[:, cut[0]] @ Wt[cut[1]] + dz[:, cut[1]] @ Wt[cut[0]]})
    else:
        wrong["slope of one"] = dY @ Wt
        parts.append(exact - dY @ Wt)
    found = set()
    for part in parts:
        step = np.sign(part)
        ends = []
        for sign in (1, -1):
            t = dict(s, X=torch.from_numpy(X + sign * h * step).to(BF))
            ends.append((f64(t["X"]), f64(run_linear(m, t)["Y"])))
        (xa, ya), (xb, yb) = ends
        seen = ((ya - yb) * dY).sum()
        noise = ROUNDINGS * 2.0 ** -8 * np.sqrt((ya ** 2 * dY ** 2).sum() + (yb ** 2 * dY ** 2).sum())
        curve = abs(((ref.act(xa @ Wt.T + bias, act) - ref.act(xb @ Wt.T + bias, act)) * dY).sum() - (exact * (xa - xb)).sum())
        # the checkpoint's share; dZ's roundings and dX's
        kept_share = abs(((kept - dz) @ Wt * (xa - xb)).sum())
        own = ROUNDINGS * 2.0 ** -8 * np.sqrt(((kept * ((xa - xb) @ Wt.T)) ** 2).sum() + ((kept @ Wt * (xa - xb)) ** 2).sum())
        slack = noise + curve + kept_share + own
        assert abs((dX * (xa - xb)).sum() - seen) <= slack
        found |= {k for k, v in wrong.items() if abs((v * (xa - xb)).sum() - seen) > slack}
    assert found == set(wrong)


# ------------------------------------------------------------------ together

def _block(M, D, F):
    """A pre-norm feed-forward block on 8-bit rows: its layers and everything that they keep."""
    new = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    L = {"norm": _norm(M, D), "pack": _norm(M, F, "none"), "up": layer(M, D, F, "swiglu", "e4m3"),
         "down": layer(M, F, D, "none", "e4m3")}
    t = {"S": new(BF, M, D), "Q": new(F8, M, D), "Qs": new(F32, M), "Zq": new(F8, M, 2 * F), "Ze": new(torch.uint8, M, 2, -(-F // 32)),
         "H": new(BF, M, F), "Hq": new(F8, M, F), "Hs": new(F32, M), "Y": new(BF, M, D), "dH": new(BF, M, F), "dN": new(BF, M, D),
         "dW1": new(BF, 2 * F, D), "dW2": new(BF, D, F), "dS": new(BF, M, D), "dw": new(BF, D),
         "work": new(torch.uint8, max(L["up"].info.grad_work_bytes, L["down"].info.grad_work_bytes, L["norm"].info.grad_work_bytes))}
    return L, t


def _forward(L, t, p):
    L["norm"].run(p["X"], p["R"], p["w"], S=t["S"], Q=t["Q"], Qs=t["Qs"])
    L["up"].run(t["Q"], p["W1q"], t["work"], t["H"], Xs=t["Qs"], Ws=p["W1s"], Zq=t["Zq"], Ze=t["Ze"])
    L["pack"].run(t["H"], Q=t["Hq"], Qs=t["Hs"])
    L["down"].run(t["Hq"], p["W2q"], t["work"], t["Y"], Xs=t["Hs"], Ws=p["W2s"], R=t["S"])


def _backward(L, t, p):
    L["down"].run_grad(t["Hq"], p["W2"], p["dY"], t["work"], t["dH"], t["dW2"], Xs=t["Hs"])
    L["up"].run_grad(t["Q"], p["W1"], t["dH"], t["work"], t["dN"], t["dW1"], Xs=t["Qs"], Zq=t["Zq"], Ze=t["Ze"])
    L["norm"].run_grad(t["S"], p["w"], t["dN"], p["dY"], t["work"], t["dS"], t["dw"])


def _parameters(M, D, F, seed=0):
    from linear_helpers import rows8
    g = torch.Generator().manual_seed(seed)
    p = {"X": torch.randn(M, D, generator=g).to(BF), "R": torch.randn(M, D, generator=g).to(BF),
         "w": (1 + 0.2 * torch.randn(D, generator=g)).to(BF), "W1": (torch.randn(2 * F, D, generator=g) * D ** -0.5).to(BF),
         "W2": (torch.randn(D, F, generator=g) * F ** -0.5).to(BF), "dY": torch.randn(M, D, generator=g).to(BF)}
    p["W1q"], p["W1s"] = rows8(p["W1"].float())
    p["W2q"], p["W2s"] = rows8(p["W2"].float())
    return cuda(p)


@pytest.mark.parametrize("M", [1, 48, 1500])
def test_feed_forward_block(M):
    """Norm, gated product with its checkpoint, 8-bit rows, product with the residual, and all of it
    backward: each step against the oracle on the device's own inputs of that step."""
    D, F = 1024, 784
    p = _parameters(M, D, F)
    L, t = _block(M, D, F)
    _forward(L, t, p)
    _backward(L, t, p)
    assert L["up"].check(t["work"])[0] == cs.OK
    S, y = ref.norm(f64(p["X"]), f64(p["R"]), f64(p["w"]), EPS)
    assert_within(t["S"], S, 2.0 ** -8 * np.abs(S) * 1.001, "S")
    assert_rows8(t["Q"], t["Qs"], y, ref.norm_bound(S, y), "Q")
    H, bound, z, dz = ref.linear(f64(t["Q"]), f64(t["Qs"]), f64(p["W1q"]), f64(p["W1s"]), None, None, "swiglu")
    assert_within(t["H"], H, bound, "H")
    assert_checkpoint(t["Zq"], t["Ze"], z, dz, 2, "Z")
    assert_rows8(t["Hq"], t["Hs"], f64(t["H"]), 0 * H, "Hq")
    Y, bound, _, _ = ref.linear(f64(t["Hq"]), f64(t["Hs"]), f64(p["W2q"]), f64(p["W2s"]), None, f64(t["S"]), "none")
    assert_within(t["Y"], Y, bound, "Y")
    g = ref.linear_grad(f64(t["Hq"]), f64(t["Hs"]), f64(p["W2"]), None, f64(p["dY"]), "none")
    assert_within(t["dH"], *g["dX"], "dH")
    assert_within(t["dW2"], *g["dWt"], "dW2")
    zz = f64(t["Zq"]) * ref.units(t["Ze"].cpu().numpy().astype(int), 2, F)
    g = ref.linear_grad(f64(t["Q"]), f64(t["Qs"]), f64(p["W1"]), zz, f64(t["dH"]), "swiglu")
    assert_within(t["dN"], *g["dX"], "dN")
    assert_within(t["dW1"], *g["dWt"], "dW1")
    g = ref.norm_grad(f64(t["S"]), f64(p["w"]), f64(t["dN"]), f64(p["dY"]), EPS)
    assert_within(t["dS"], *g["dX"], "dS")
    assert_within(t["dw"], *g["dw"], "dw")


OUTS = ("S", "Q", "Qs", "Zq", "Ze", "H", "Y", "dH", "dN", "dW1", "dW2", "dS", "dw")


@pytest.mark.parametrize("M", [1, 48, 1500])
def test_same_bytes_every_time_and_from_a_graph(M):
    D, F = 1024, 784
    p = _parameters(M, D, F)
    L, t = _block(M, D, F)
    _forward(L, t, p)
    _backward(L, t, p)
    want = {k: t[k].clone() for k in OUTS}

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(t[k].view(torch.uint8), want[k].view(torch.uint8)) for k in OUTS)
    for _ in range(3):
        _forward(L, t, p)
        _backward(L, t, p)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _forward(L, t, p)
        _backward(L, t, p)
    for _ in range(3):
        for k in OUTS:
            t[k].view(torch.uint8).fill_(0x55)
        graph.replay()
        assert same()
    # new inputs through the same graph
    q = _parameters(M, D, F, seed=1)
    for k in p:
        p[k].copy_(q[k])
    graph.replay()
    torch.cuda.synchronize()
    got = {k: t[k].clone() for k in OUTS}
    _forward(L, t, p)
    _backward(L, t, p)
    assert all(torch.equal(t[k].view(torch.uint8), got[k].view(torch.uint8)) for k in OUTS)


def test_calls_side_by_side():
    """Two blocks on two streams at once, with buffers of their own."""
    D, F, sizes = 1024, 784, (64, 1300)
    ps, blocks, streams, wants = [], [], [], []
    for i, M in enumerate(sizes):
        ps.append(_parameters(M, D, F, seed=i))
        blocks.append(_block(M, D, F))
        _forward(*blocks[i], ps[i])
        _backward(*blocks[i], ps[i])
        wants.append({k: blocks[i][1][k].clone() for k in OUTS})
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                _forward(*blocks[i], ps[i])
                _backward(*blocks[i], ps[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(blocks[i][1][k].view(torch.uint8), wants[i][k].view(torch.uint8)) for k in OUTS)
        assert blocks[i][0]["up"].check(blocks[i][1]["work"])[0] == cs.OK


@pytest.mark.parametrize("M", [40, 1300])
def test_one_graph_after_another_with_one_buffer(M):
    """Two captured passes that share a work buffer, replayed in order on one stream; a capture behind other work."""
    K, N = 1000, 776
    s = [linear_inputs(M, K, N, "gelu", "bf16", seed=i, grad=True) for i in (1, 2)]
    m = layer(M, K, N, "gelu")
    want = [run_linear_grad(m, x) for x in s]
    work = torch.empty(m.info.grad_work_bytes, dtype=torch.uint8, device="cuda")
    d = [cuda(x) for x in s]
    out = [{k: torch.zeros_like(v) for k, v in w.items()} for w in want]
    graphs = []
    for x, o in zip(d, out):
        g = torch.cuda.CUDAGraph()
        torch.cuda._sleep(1000000)
        with torch.cuda.graph(g):
            m.run_grad(x["X"], x["Wt"], x["dY"], work, o["dX"], o["dWt"], o["dbias"], Zq=x["Zq"], Ze=x["Ze"])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        assert all(torch.equal(o[k], w[k]) for k in w)
    assert m.check(work)[0] == cs.OK


FRESH = r"""
import sys, torch
import tile_level_sync_gb300 as cs
first = sys.argv[1]
bf, f8 = torch.bfloat16, torch.float8_e4m3fn
new = lambda dtype, *shape: torch.ones(shape, dtype=torch.float32, device="cuda").to(dtype)
M = 3
n = cs.Norm(cs.make_norm_desc(M=M, D=64))
if first == "norm": n.run(new(bf, M, 64), None, new(bf, 64), Y=new(bf, M, 64))
if first == "linear":
    m = cs.Linear(cs.make_linear_desc(M=M, K=64, N=64))
    m.run(new(bf, M, 64), new(bf, 64, 64), new(torch.uint8, m.info.work_bytes), new(bf, M, 64))
for M, D in ((5, 264), (1100, 264), (5, 12288), (5, 20480)):
    n = cs.Norm(cs.make_norm_desc(M=M, D=D))
    x, w, y, dx, dw, work = new(bf, M, D), new(bf, D), new(bf, M, D), new(bf, M, D), new(bf, D), new(torch.uint8, n.info.grad_work_bytes)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n.run(x, None, w, Y=y)
        n.run_grad(x, w, y, None, work, dx, dw)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, dx, dw)]
    n.run(x, None, w, Y=y)
    n.run_grad(x, w, y, None, work, dx, dw)
    assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw)))
for M, K, N, act in ((20, 256, 264, "gelu"), (1300, 528, 2056, "swiglu"), (2048, 1024, 2048, "relu")):
    m = cs.Linear(cs.make_linear_desc(M=M, K=K, N=N, act=act))
    G = m.info.parts
    x, W, dy, y = new(bf, M, K), new(bf, G * N, K), new(bf, M, N), new(bf, M, N)
    Zq, Ze = new(f8, M, G * N), new(torch.uint8, M, G, m.info.blocks)
    dx, dW, db, work = new(bf, M, K), new(bf, G * N, K), new(bf, G * N), new(torch.uint8, m.info.grad_work_bytes)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.run(x, W, work, y, Zq=Zq, Ze=Ze)
        m.run_grad(x, W, dy, work, dx, dW, db, Zq=Zq, Ze=Ze)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, dx, dW, db)]
    m.run(x, W, work, y, Zq=Zq, Ze=Ze)
    m.run_grad(x, W, dy, work, dx, dW, db, Zq=Zq, Ze=Ze)
    assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dW, db)))
print("same bytes")
"""


@pytest.mark.parametrize("first", ["none", "norm", "linear"])
def test_captures_in_a_fresh_process(first):
    """Captures of calls whose kernels no call has launched before them, and whose attributes another call has set, or none."""
    r = subprocess.run([sys.executable, "-c", FRESH, first], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "same bytes" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_calls_beside_other_kernels_of_the_library():
    """A layer of experts on one stream and linear layers on another, which share the SMs' tensor memory."""
    from moe_helpers import layer as experts, mlp_inputs
    x = mlp_inputs(700, 8, 2, 1024, 512, "swiglu")
    moe, dx = experts(x, "swiglu"), {k: v.cuda() for k, v in x.items()}
    mwork, Y = torch.empty(moe.info.work_bytes, dtype=torch.uint8, device="cuda"), torch.empty_like(dx["X"])
    moe.mlp(dx["X"], dx["W1t"], dx["W2t"], dx["ids"], dx["weights"], mwork, Y)
    want = Y.clone()
    layers = []
    for M, K, N in ((20, 1024, 1032), (1300, 520, 2056), (200, 4096, 264)):
        s = linear_inputs(M, K, N, "swiglu")
        m = layer(M, K, N, "swiglu")
        layers.append((m, cuda(s), torch.empty(m.info.work_bytes, dtype=torch.uint8, device="cuda"),
                       torch.empty(M, N, dtype=BF, device="cuda"), run_linear(m, s)["Y"]))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(a):
            moe.mlp(dx["X"], dx["W1t"], dx["W2t"], dx["ids"], dx["weights"], mwork, Y)
        with torch.cuda.stream(b):
            for m, d, work, y, _ in layers:
                m.run(d["X"], d["Wt"], work, y, bias=d["bias"], R=d["R"])
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and moe.check(mwork)[0] == cs.OK
    for m, d, work, y, w in layers:
        assert torch.equal(y, w) and m.check(work)[0] == cs.OK


def test_no_rows():
    e = lambda *shape, dtype=BF: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    n = _norm(0, 64)
    n.run(e(0, 64), None, e(64), Y=e(0, 64))
    dw = torch.full((64,), 3.0, dtype=BF, device="cuda")
    n.run_grad(e(0, 64), e(64), e(0, 64), None, e(n.info.grad_work_bytes, dtype=torch.uint8), e(0, 64), dw)
    assert (dw == 0).all()
    m = layer(0, 64, 72, "swiglu")
    work = torch.full((m.info.grad_work_bytes,), 0x77, dtype=torch.uint8, device="cuda")
    m.run(e(0, 64), e(144, 64), work, e(0, 72))
    assert m.check(work) == (cs.OK, 0)
    work.fill_(0x77)
    dWt, db = torch.full((144, 64), 3.0, dtype=BF, device="cuda"), torch.full((144,), 3.0, dtype=BF, device="cuda")
    m.run_grad(e(0, 64), e(144, 64), e(0, 72), work, e(0, 64), dWt, db, Zq=e(0, 144, dtype=F8), Ze=e(0, 2, 3, dtype=torch.uint8))
    assert (dWt == 0).all() and (db == 0).all() and m.check(work) == (cs.OK, 0)


def test_check_is_refused_in_a_capture():
    m = layer(4, 64, 64, "none")
    work = torch.zeros(m.info.work_bytes, dtype=torch.uint8, device="cuda")
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.run(x, x.new_zeros(64, 64), work, torch.empty_like(x))
        try:
            status = m.check(work)[0]
        except cs.CusyncError as e:
            status = e.status
    assert status == cs.ERR_UNSUPPORTED
    graph.replay()
    assert m.check(work) == (cs.OK, 0)


# ------------------------------------------------------------------ long tensors

def test_norm_offsets_beyond_32_bits():
    M, D = (1 << 31) // 8192 + 40, 8192
    x = torch.zeros(M, D, dtype=BF, device="cuda")
    s = norm_inputs(16, D)
    x[-16:] = s["X"].cuda()
    w, Q, Qs = s["w"].cuda(), torch.empty(M, D, dtype=F8, device="cuda"), torch.empty(M, device="cuda")
    n = _norm(M, D)
    n.run(x, None, w, Q=Q, Qs=Qs)
    S, y = ref.norm(f64(s["X"]), None, f64(s["w"]), EPS)
    assert_rows8(Q[-16:], Qs[-16:], y, ref.norm_bound(S, y), "Q")
    assert (Q[:1000].float() == 0).all()
    dY, work, dw = torch.zeros_like(x), torch.empty(n.info.grad_work_bytes, dtype=torch.uint8, device="cuda"), torch.empty_like(w)
    dY[-16:] = s["dY"].cuda()
    dX = torch.empty_like(x)
    n.run_grad(x, w, dY, None, work, dX, dw)
    want = ref.norm_grad(f64(s["X"]), f64(s["w"]), f64(s["dY"]), None, EPS)
    assert_within(dX[-16:], *want["dX"], "dX")
    assert_within(dw, *want["dw"], "dw")


def test_linear_offsets_beyond_32_bits():
    M, K, N = (1 << 31) // 2048 // 2 + 1300, 64, 2048   # the checkpoint's and dZ's 2 N columns
    s = linear_inputs(16, K, N, "swiglu", residual=False)
    X = torch.zeros(M, K, dtype=BF, device="cuda")
    X[-16:] = s["X"].cuda()
    d = cuda(s)
    m = layer(M, K, N, "swiglu")
    Zq, Ze = torch.empty(M, 2 * N, dtype=F8, device="cuda"), torch.empty(M, 2, N // 32, dtype=torch.uint8, device="cuda")
    Y, work = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(m.info.grad_work_bytes, dtype=torch.uint8, device="cuda")
    m.run(X, d["Wt"], work, Y, bias=d["bias"], Zq=Zq, Ze=Ze)
    want, bound, z, dz = oracle_linear(s, "swiglu")
    assert_within(Y[-16:], want, bound, "Y")
    assert_checkpoint(Zq[-16:], Ze[-16:], z, dz, 2, "Z")
    dY = torch.zeros(M, N, dtype=BF, device="cuda")
    dY[-16:] = d["dY"]
    dX, dWt, db = torch.empty_like(X), torch.empty_like(d["Wt"]), torch.empty_like(d["bias"])
    m.run_grad(X, d["Wt"], dY, work, dX, dWt, db, Zq=Zq, Ze=Ze)
    assert m.check(work)[0] == cs.OK
    s.update(Zq=Zq[-16:].cpu(), Ze=Ze[-16:].cpu())
    g = oracle_grad(s, "swiglu")
    assert_within(dX[-16:], *g["dX"], "dX")
    assert_within(dWt, *g["dWt"], "dWt")
    assert_within(db, *g["dbias"], "dbias")


def test_tall_residuals_beyond_32_bits():
    M, K, N = 140000, 16, 16392
    s = linear_inputs(16, K, N, "none")
    X, R = torch.zeros(M, K, dtype=BF, device="cuda"), torch.zeros(M, N, dtype=BF, device="cuda")
    X[-16:], R[-16:] = s["X"].cuda(), s["R"].cuda()
    d, m = cuda(s), layer(M, K, N, "none")
    m.run(X, d["Wt"], torch.empty(m.info.work_bytes, dtype=torch.uint8, device="cuda"), R, bias=d["bias"], R=R)
    want, bound, _, _ = oracle_linear(s, "none")
    assert_within(R[-16:], want, bound, "Y")
    assert torch.equal(R[5], d["bias"])
