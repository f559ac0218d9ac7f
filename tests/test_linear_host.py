"""CPU tests of the norm and linear layers: the oracle's pins, buffer sizes, refusals and the
binding."""

import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import tile_level_sync_gb300 as cs
from oracle import linear as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ the oracle

def test_oracle_e4m3_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 1, 20000) * 2.0 ** rng.integers(-12, 9, 20000), np.arange(-448, 449) / 2,
                        [2.0 ** -10, 1.5 * 2.0 ** -9, 2.0 ** -11, 17.0, 19.0, 0.0]])
    x = np.clip(x.astype(np.float32), -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.round_to_e4m3(x), want)


def test_oracle_norm_by_hand():
    X, R, w = np.array([[3.0, 0.0]]), np.array([[0.0, 4.0]]), np.array([1.0, 2.0])
    S, y = ref.norm(X, R, w, 0.0)
    assert S.tolist() == [[3.0, 4.0]] and np.allclose(y, [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]])
    assert np.allclose(ref.row_scales(y), [8 / 12.5 ** 0.5 / 448])
    assert ref.row_scales(np.array([[0.0, np.inf], [1.0, np.nan]])).tolist() == [2.0 ** -126, 1 / 448]


def test_oracle_exponents():
    z = np.array([[448.0, 1.0] + [0.0] * 30 + [448.1] + [0.0] * 7, [0.0] * 32 + [1e-40] * 8,
                  [224.0] * 32 + [np.inf, 225.0] + [0.0] * 6])
    assert ref.exponents(z, 1)[:, 0].tolist() == [[127, 128], [1, 1], [126, 127]]
    assert ref.exponents(z, 2).shape == (3, 2, 1)
    q, e = ref.checkpoint(np.array([[896.0, 1.0]]), 1)
    assert q.tolist() == [[448.0, 0.5]] and e.tolist() == [[[128]]]


def _differences(f, arg, got, tol=1e-6, h=1e-6):
    for i in np.ndindex(arg.shape):
        keep, d = arg[i], []
        for x in (h, -h):
            arg[i] = keep + x
            d.append(f())
        arg[i] = keep
        assert abs(got[i] - (d[0] - d[1]) / (2 * h)) < tol, i


def test_oracle_norm_grad_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    S, w, dY, dS = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    g = ref.norm_grad(S, w, dY, dS, 1e-3)
    f = lambda: (ref.norm(S, None, w, 1e-3)[1] * dY).sum() + (S * dS).sum()  # noqa: E731
    _differences(f, S, g["dX"][0])
    _differences(f, w, g["dw"][0])


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
def test_oracle_linear_grad_is_the_difference_quotient(act):
    rng = np.random.default_rng(2)
    G = 2 if act == "swiglu" else 1
    X, Wt, bias, dY = rng.normal(size=(4, 3)), rng.normal(size=(5 * G, 3)), rng.normal(size=5 * G), rng.normal(size=(4, 5))
    z = X @ Wt.T + bias
    f = lambda: (ref.act(X @ Wt.T + bias, act) * dY).sum()  # noqa: E731
    dz, _ = ref.slope(z, dY, act)
    _differences(f, X, dz @ Wt)
    _differences(f, Wt, dz.T @ X)
    _differences(f, bias, dz.sum(axis=0))
    # the gradients of linear_grad: the same up to dZ's rounding to bf16
    for name, want in (("dX", dz @ Wt), ("dWt", dz.T @ X), ("dbias", dz.sum(axis=0))):
        got, bound = ref.linear_grad(X, None, Wt, None if act == "none" else z, dY, act)[name]
        assert np.all(bound >= 0) and np.allclose(got, want, atol=0.2, rtol=0.02), name
        # rows of 8 bits: the same for their values
        Xs = np.array([0.3, 1.0, 1.7, 5.0])
        again, _ = ref.linear_grad(X / Xs[:, None], Xs, Wt, None if act == "none" else z, dY, act)[name]
        assert np.allclose(again, want, atol=0.2, rtol=0.02), name


def test_oracle_slopes_of_nan_are_nan():
    z, dY = np.array([[np.nan, 2.0, -2.0, 1.0, 1.0, 1.0]]), np.full((1, 6), 3.0)
    for act in ("relu", "gelu"):
        dz = ref.slope(z, dY, act)[0]
        assert np.isnan(dz[0, 0]) and np.isfinite(dz[0, 1:]).all()
    assert ref.slope(z, dY, "relu")[0][0, 1:].tolist() == [3.0, 0.0, 3.0, 3.0, 3.0]
    with np.errstate(invalid="ignore"):
        gated = ref.slope(z, dY[:, :3], "swiglu")[0]
    assert np.isnan(gated).tolist() == [[True, False, False, True, False, False]]


# ------------------------------------------------------------------ header and binding

def _header():
    src = open(os.path.join(ROOT, "include", "cusync_linear.h")).read()
    return re.sub(r"/\*.*?\*/", "", src, flags=re.S)


def test_library_exports_every_declared_function():
    names = re.findall(r"\bcusync_status_t\s+(cusync_\w+)\s*\(", _header())
    assert len(names) == 7
    assert all(hasattr(cs.load(), n) for n in names)


def test_binding_constants_match_header():
    src = _header()
    vals = {k: int(v) for k, v in re.findall(r"\bCUSYNC_(\w+)\s*=\s*(\d+)", src)}
    vals.update({k: int(v) for k, v in re.findall(r"#define\s+CUSYNC_(\w+)\s+(\d+)\s*$", src, flags=re.M)})
    assert len(vals) == 10
    for name, v in vals.items():
        assert getattr(cs, name) == v, name


# ------------------------------------------------------------------ sizes and refusals

NORM = dict(M=10, D=64)
LINEAR = dict(M=10, K=64, N=96)


def _status(f):
    try:
        f()
    except cs.CusyncError as e:
        return e.status
    return cs.OK


@pytest.mark.parametrize("change,status", [
    (dict(), cs.OK), (dict(M=0), cs.OK), (dict(D=8), cs.OK), (dict(D=32768), cs.OK), (dict(kind="none"), cs.OK),
    (dict(eps=0.0), cs.OK), (dict(M=-1), cs.ERR_INVALID_ARG), (dict(D=0), cs.ERR_INVALID_ARG),
    (dict(kind=2), cs.ERR_INVALID_ARG), (dict(eps=-1e-6), cs.ERR_INVALID_ARG), (dict(eps=float("nan")), cs.ERR_INVALID_ARG),
    (dict(eps=float("inf")), cs.ERR_INVALID_ARG), (dict(num_sms=-1), cs.ERR_INVALID_ARG), (dict(D=12), cs.ERR_UNSUPPORTED),
    (dict(D=32776), cs.ERR_UNSUPPORTED), (dict(M=1 << 31), cs.ERR_UNSUPPORTED),
])
def test_norm_descriptors(change, status):
    assert _status(lambda: cs.cusync_norm_info(cs.make_norm_desc(**{**NORM, **change}))) == status


@pytest.mark.parametrize("change,status", [
    (dict(), cs.OK), (dict(M=0), cs.OK), (dict(K=8, N=8), cs.OK), (dict(dtype="e4m3"), cs.OK), (dict(act="swiglu"), cs.OK),
    (dict(M=-1), cs.ERR_INVALID_ARG), (dict(K=0), cs.ERR_INVALID_ARG), (dict(N=0), cs.ERR_INVALID_ARG),
    (dict(act=4), cs.ERR_INVALID_ARG), (dict(act=-1), cs.ERR_INVALID_ARG), (dict(dtype=2), cs.ERR_INVALID_ARG),
    (dict(num_sms=-1), cs.ERR_INVALID_ARG), (dict(K=12), cs.ERR_UNSUPPORTED), (dict(N=12), cs.ERR_UNSUPPORTED),
    (dict(K=8, dtype="e4m3"), cs.ERR_UNSUPPORTED), (dict(K=1 << 25), cs.ERR_UNSUPPORTED), (dict(N=1 << 25), cs.ERR_UNSUPPORTED),
    (dict(M=(1 << 30) + 1), cs.ERR_UNSUPPORTED), (dict(M=1 << 30, N=1 << 20), cs.ERR_UNSUPPORTED),
])
def test_linear_descriptors(change, status):
    assert _status(lambda: cs.cusync_linear_info(cs.make_linear_desc(**{**LINEAR, **change}))) == status


def test_sizes():
    assert cs.cusync_norm_info(cs.make_norm_desc(**NORM)).grad_work_bytes >= 64 * 4 * 10
    i = cs.cusync_linear_info(cs.make_linear_desc(M=10, K=64, N=104, act="swiglu", dtype="e4m3"))
    assert (i.parts, i.blocks) == (2, 4)
    # dZ, X in bf16 and the bias's partial sums
    assert i.work_bytes >= 4 and i.grad_work_bytes >= i.work_bytes + 10 * 208 * 2 + 10 * 64 * 2 + 208 * 4
    small = cs.cusync_linear_info(cs.make_linear_desc(M=10, K=64, N=104))
    assert small.parts == 1 and small.grad_work_bytes < i.grad_work_bytes


def test_null_and_misaligned_pointers_are_refused():
    """Refused before anything is launched: this runs without a GPU."""
    import ctypes
    lib, P = cs.load(), 4096
    n, nd = ctypes.byref(cs.make_norm_desc(**NORM)), ctypes.byref(cs.make_norm_desc(**NORM, kind="none"))

    def norm(d=n, X=P, R=None, w=P, S=P, Y=P, Q=P, Qs=P):
        return lib.cusync_norm(d, X, R, w, S, Y, Q, Qs, None)
    for bad in (dict(X=None), dict(X=P + 8), dict(w=None), dict(R=P + 2), dict(S=P + 4), dict(Y=P + 8), dict(Q=P + 8),
                dict(Q=None), dict(Qs=None), dict(Qs=P + 4), dict(S=None, Y=None, Q=None, Qs=None), dict(d=None)):
        assert norm(**bad) == cs.ERR_INVALID_ARG, bad

    def norm_grad(d=n, S=P, w=P, dY=P, dS=P, work=P, dX=P, dw=P):
        return lib.cusync_norm_grad(d, S, w, dY, dS, work, dX, dw, None)
    for name in ("S", "w", "dY", "work", "dX"):
        assert norm_grad(**{name: None}) == cs.ERR_INVALID_ARG, name
    for name in ("S", "w", "dY", "dS", "work", "dX", "dw"):
        assert norm_grad(**{name: P + 8}) == cs.ERR_INVALID_ARG, name
    assert norm_grad(d=nd) == cs.ERR_UNSUPPORTED

    b, f = ctypes.byref(cs.make_linear_desc(**LINEAR, act="gelu")), ctypes.byref(cs.make_linear_desc(**LINEAR, dtype="e4m3"))

    def linear(d=b, X=P, Xs=None, Wt=P, Ws=None, bias=None, R=None, work=P, Y=P, Zq=None, Ze=None):
        return lib.cusync_linear(d, X, Xs, Wt, Ws, bias, R, work, Y, Zq, Ze, None)
    for bad in (dict(X=None), dict(Wt=None), dict(work=None), dict(Y=None), dict(Xs=P), dict(Ws=P), dict(Zq=P), dict(Ze=P),
                dict(X=P + 8), dict(Wt=P + 8), dict(bias=P + 2), dict(R=P + 2), dict(work=P + 4), dict(Y=P + 2),
                dict(Zq=P + 8, Ze=P), dict(Zq=P, Ze=P + 1), dict(d=f), dict(d=f, Xs=P), dict(d=f, Ws=P), dict(d=None)):
        assert linear(**bad) == cs.ERR_INVALID_ARG, bad

    def grad(d=b, X=P, Xs=None, Wt=P, Zq=P, Ze=P, dY=P, work=P, dX=P, dWt=P, dbias=P):
        return lib.cusync_linear_grad(d, X, Xs, Wt, Zq, Ze, dY, work, dX, dWt, dbias, None)
    for name in ("X", "Wt", "Zq", "Ze", "dY", "work"):
        assert grad(**{name: None}) == cs.ERR_INVALID_ARG, name
    for name in ("X", "Wt", "Zq", "Ze", "dY", "work", "dX", "dWt", "dbias"):
        assert grad(**{name: P + 8}) == cs.ERR_INVALID_ARG, name
    for bad in (dict(dX=None, dWt=None, dbias=None), dict(Xs=P), dict(d=f, Zq=None, Ze=None), dict(d=None)):
        assert grad(**bad) == cs.ERR_INVALID_ARG, bad
    assert lib.cusync_linear_check(None, None, None) == cs.ERR_INVALID_ARG
    assert lib.cusync_linear_check(P + 4, None, None) == cs.ERR_INVALID_ARG


def test_binding_checks_tensors():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    n = cs.Norm(cs.make_norm_desc(**NORM))
    x, w = torch.zeros(10, 64, dtype=bf), torch.zeros(64, dtype=bf)
    with pytest.raises(ValueError, match="X is torch.float32"):
        n.run(x.float(), None, w, Y=x)
    with pytest.raises(ValueError, match="w has 63 elements"):
        n.run(4096, None, w[:63], Y=4096)
    with pytest.raises(ValueError, match="Y is not contiguous"):
        n.run(4096, None, 4096, Y=torch.zeros(64, 10, dtype=bf).t())
    with pytest.raises(ValueError, match="Q is torch.uint8"):
        n.run(4096, None, 4096, Q=torch.zeros(10, 64, dtype=torch.uint8), Qs=4096)
    with pytest.raises(ValueError, match="on cpu"):
        n.run(x, None, w, Y=x)
    with pytest.raises(ValueError, match="work holds 8 bytes"):
        n.run_grad(4096, 4096, 4096, None, torch.zeros(2), 4096, 4096)
    m = cs.Linear(cs.make_linear_desc(**LINEAR, act="swiglu", dtype="e4m3"))
    with pytest.raises(ValueError, match="Wt is torch.bfloat16"):
        m.run(4096, torch.zeros(192, 64, dtype=bf), 4096, 4096, Xs=4096, Ws=4096)
    with pytest.raises(ValueError, match="Wt has 6144 elements"):
        m.run(4096, torch.zeros(96, 64).to(f8), 4096, 4096, Xs=4096, Ws=4096)
    with pytest.raises(ValueError, match="Ze has 30 elements: 60"):
        m.run(4096, 4096, 4096, 4096, Xs=4096, Ws=4096, Zq=4096, Ze=torch.zeros(10, 3, dtype=torch.uint8))
    with pytest.raises(ValueError, match="Wt is torch.float8_e4m3fn: torch.bfloat16"):
        m.run_grad(4096, torch.zeros(192, 64).to(f8), 4096, 4096, 4096, 4096, Xs=4096, Zq=4096, Ze=4096)
    with pytest.raises(cs.CusyncError):
        m.run(4096, 4096, 4096, 4096, stream=0)  # without scales
    with pytest.raises(KeyError):
        cs.make_linear_desc(**LINEAR, act="tanh")


PLANNER = r"""
#include <cstdio>
#include "lin_plan.h"
using namespace cusync::lin;
int bad = 0, seen = 0;
template <int MODE, bool GATED>
void look(int64_t rows, int64_t cols, int64_t depth, int sms, int elems) {
  const Plan s = split_plan<MODE, GATED>(rows, cols, depth, sms, elems), p = pair_plan(rows, cols, depth, sms, elems, GATED);
  const bool pow2 = (s.cols & (s.cols - 1)) == 0 && (s.splits & (s.splits - 1)) == 0;
  const int64_t stages = (div_up(depth, elems) + 1) / 2;
  // nothing takes less than its start and end; a CTA has a stage of the reduction at least
  const bool ok = s.us >= 5.2 && s.us < 1e12 && pow2 && s.cols >= (MODE == DW ? 64 : 16) && s.cols <= 128 && s.splits >= 1 &&
                  s.splits <= 8 && s.splits <= stages && s.stages >= 1 && s.stages <= kMaxStages && s.stages * s.splits <= stages + s.splits - 1 &&
                  split_smem(s.cols, s.stages, s.apart) <= (size_t)kSmemPerSm - 1024 &&
                  (sms < 2 ? p.us == 1e30 && !p.bn : p.us >= 4.2 && p.us < 1e12 && (p.bn == 128 || p.bn == 256));
  ++seen;
  if (!ok) ++bad, std::printf("mode %d gated %d %lld x %lld x %lld on %d: %g us, %d, %d, %d\n", MODE, GATED, (long long)rows,
                              (long long)cols, (long long)depth, sms, s.us, s.cols, s.splits, s.stages);
}
int main() {
  const int64_t sizes[] = {1, 8, 20, 64, 72, 100, 333, 776, 1000, 1281, 2056, 9000};
  for (int sms : {1, 2, 3, 4, 5, 6, 7, 8, 37, 151, 152})
    for (int64_t rows : sizes)
      for (int64_t cols : sizes)
        for (int64_t depth : sizes) {
          look<FWD, false>(rows, cols, depth, sms, 64);
          look<FWD, false>(rows, cols, depth, sms, 128);
          look<FWD, true>(rows, cols, depth, sms, 64);
          look<FWD, true>(rows, cols, depth, sms, 128);
          look<DX, false>(rows, cols, depth, sms, 64);
          look<DW, false>(rows, cols, depth, sms, 64);
        }
  std::printf("%d plans, %d bad\n", seen, bad);
  return bad != 0;
}
"""


def test_plans_on_any_number_of_sms(tmp_path):
    """The plans of all kinds of products are sound from one SM on; a division by zero traps, whatever the host makes of one."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    src = tmp_path / "plans.cpp"
    src.write_text(PLANNER)
    build = subprocess.run([gxx, "-std=c++17", "-O1", "-fsanitize=integer-divide-by-zero", "-fsanitize-undefined-trap-on-error",
                            "-I" + os.path.join(ROOT, "tile_level_sync_gb300", "csrc_linear"), str(src), "-o", str(tmp_path / "plans")],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    r = subprocess.run([str(tmp_path / "plans")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout[-2000:])
    assert int(r.stdout.split()[0]) > 100000
