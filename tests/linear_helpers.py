"""Inputs and runs of the norm and linear layers' tests."""

import numpy as np
import torch

import tile_level_sync_gb300 as cs
from oracle import linear as ref

BF, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


def f64(t):
    return None if t is None else t.detach().cpu().float().double().numpy()


class Out:
    """A device tensor, filled with NaN, with 4 KB of a known pattern behind it."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        self.buf[n:] = 0x5A
        self.t = self.buf[:n].view(dtype).view(shape) if n else torch.empty(shape, dtype=dtype, device="cuda")

    def intact(self):
        return bool((self.buf[-4096:] == 0x5A).all())


def rows8(y, seed=0):
    """8-bit rows of y (fp32 CPU tensor)."""
    s = (y.abs().amax(dim=1) / 448).clamp(min=2.0 ** -126)
    return (y / s[:, None]).clamp(-448, 448).to(F8), s


def norm_inputs(M, D, residual=True, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * M + D)
    rows = torch.exp(2 * torch.randn(M, 1, generator=g))
    s = {"X": (rows * torch.randn(M, D, generator=g)).to(BF), "w": (1 + 0.3 * torch.randn(D, generator=g)).to(BF),
         "R": (rows * torch.randn(M, D, generator=g)).to(BF) if residual else None,
         "dY": torch.randn(M, D, generator=g).to(BF)}
    return s


def linear_inputs(M, K, N, act, dtype="bf16", bias=True, residual=True, seed=0, grad=False):
    g = torch.Generator().manual_seed(seed + 7 * M + 3 * K + N)
    G = 2 if act == "swiglu" else 1
    x = torch.randn(M, K, generator=g)
    w = torch.randn(G * N, K, generator=g) * K ** -0.5 * torch.exp(0.5 * torch.randn(G * N, 1, generator=g))
    s = {"Xs": None, "Ws": None, "bias": torch.randn(G * N, generator=g).to(BF) if bias else None,
         "R": torch.randn(M, N, generator=g).to(BF) if residual else None, "dY": torch.randn(M, N, generator=g).to(BF)}
    if dtype == "e4m3":
        s["X"], s["Xs"] = rows8(x)
    else:
        s["X"] = x.to(BF)
    if dtype == "e4m3" and not grad:
        s["Wt"], s["Ws"] = rows8(w)
    else:
        s["Wt"] = w.to(BF)
    if grad and act != "none":
        z = 1.5 * torch.randn(M, G * N, generator=g)
        q, e = ref.checkpoint(z.double().numpy(), G)
        s["Zq"] = torch.from_numpy(q).float().to(F8)
        s["Ze"] = torch.from_numpy(e.astype(np.uint8))
    return s


def cuda(s):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}


def layer(M, K, N, act, dtype="bf16", **more):
    return cs.Linear(cs.make_linear_desc(M=M, K=K, N=N, act=act, dtype=dtype, **more))


def finish(m, work, outs):
    st, code = m.check(work.t)
    assert st == cs.OK, hex(code)
    assert work.intact() and all(o.intact() for o in outs)


def run_linear(m, s, checkpoint=False):
    """{"Y", "Zq", "Ze"} on the GPU; nothing behind the outputs is touched."""
    d, i, c = cuda(s), m.info, m.desc
    out = {"Y": Out((c.M, c.N), BF)}
    if checkpoint:
        out.update(Zq=Out((c.M, i.parts * c.N), F8), Ze=Out((c.M, i.parts, i.blocks), torch.uint8))
    work = Out((i.work_bytes,), torch.uint8)
    m.run(d["X"], d["Wt"], work.t, Xs=d["Xs"], Ws=d["Ws"], bias=d["bias"], R=d["R"], **{k: o.t for k, o in out.items()})
    finish(m, work, out.values())
    return {k: o.t for k, o in out.items()}


def run_linear_grad(m, s, want=("dX", "dWt", "dbias")):
    d, i, c = cuda(s), m.info, m.desc
    shapes = {"dX": (c.M, c.K), "dWt": (i.parts * c.N, c.K), "dbias": (i.parts * c.N,)}
    out = {k: Out(shapes[k], BF) for k in want}
    work = Out((i.grad_work_bytes,), torch.uint8)
    t = {k: out[k].t if k in out else None for k in shapes}
    m.run_grad(d["X"], d["Wt"], d["dY"], work.t, t["dX"], t["dWt"], t["dbias"], Xs=d["Xs"], Zq=d.get("Zq"), Ze=d.get("Ze"))
    finish(m, work, out.values())
    return {k: o.t for k, o in out.items()}


def assert_within(got, want, bound, what):
    got = f64(got).reshape(want.shape)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    worst = float(np.max(np.abs(got - want) / (bound + 1e-30))) if want.size else 0.0
    assert worst <= 1.0, f"{what}: worst error / bound = {worst:.3f}"


def assert_rows8(q, scales, y, err, what):
    """8-bit rows of y, known up to err: the scales, then each value by the device's own scale."""
    want = ref.row_scales(y)
    s = scales.detach().cpu().double().numpy()
    most = (np.abs(y) + err).max(axis=1) - np.abs(y).max(axis=1)
    assert np.all(np.abs(s - want) <= most / 448 + 3 * 2.0 ** -24 * want), f"{what}: scales"
    v = f64(q) * s[:, None]
    bound = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s[:, None]) + 2 * err + 2.0 ** -22 * np.abs(y)
    assert_within(torch.from_numpy(v), y, bound, what)


def assert_checkpoint(Zq, Ze, z, err, parts, what):
    """A checkpoint of z, known up to err: exponents that some z within err has, values by the
    device's own exponents."""
    N = z.shape[1] // parts
    e = Ze.detach().cpu().numpy().astype(int)
    low, high = ref.exponents(np.maximum(np.abs(z) - err, 0), parts), ref.exponents(np.abs(z) + err, parts)
    assert np.all((low <= e) & (e <= high)), f"{what}: exponents"
    unit = ref.units(e, parts, N)
    v = f64(Zq) * unit
    assert_within(torch.from_numpy(v), z, np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10 * unit) + 2 * err, what)


def values(s, parts):
    """What a case's checkpoint stands for."""
    if "Zq" not in s:
        return None
    return f64(s["Zq"]) * ref.units(s["Ze"].cpu().numpy().astype(int), parts, s["Zq"].shape[1] // parts)


def oracle_linear(s, act):
    return ref.linear(f64(s["X"]), f64(s["Xs"]), f64(s["Wt"]), f64(s["Ws"]), f64(s["bias"]), f64(s["R"]), act)


def oracle_grad(s, act):
    return ref.linear_grad(f64(s["X"]), f64(s["Xs"]), f64(s["Wt"]), values(s, 2 if act == "swiglu" else 1), f64(s["dY"]), act)
