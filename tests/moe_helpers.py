"""Inputs and runs of the mixture-of-experts tests."""

import numpy as np
import torch

import tile_level_sync_gb300 as cs

TINY = 1e-30  # a bound of zero still admits a denormal


def f64(t):
    return t.detach().cpu().double().numpy()


def mlp_inputs(T, E, k, D, N1, act, seed=0, ids=None):
    g = torch.Generator().manual_seed(seed)
    G = 2 if act == "swiglu" else 1
    bf = torch.bfloat16
    s = {"X": torch.randn(T, D, generator=g).to(bf), "W1t": (torch.randn(E, G * N1, D, generator=g) * D ** -0.5).to(bf),
         "W2t": (torch.randn(E, D, N1, generator=g) * N1 ** -0.5).to(bf), "dY": torch.randn(T, D, generator=g).to(bf)}
    logits = torch.randn(T, E, generator=g) + torch.randn(E, generator=g)
    s["ids"] = torch.argsort(logits, dim=1, descending=True)[:, :k].to(torch.int32).contiguous() if ids is None else ids
    s["weights"] = torch.rand(T, k, generator=g)
    return s


def layer(s, act, **more):
    T, D = s["X"].shape
    E, _, N1 = s["W2t"].shape
    return cs.Moe(cs.make_moe_desc(T=T, D=D, N1=N1, experts=E, top_k=s["ids"].shape[1], act=act, **more))


def guarded(n_bytes):
    """A device buffer of n_bytes, NaN in every type that the kernels keep there, with 4 KB of a
    known pattern behind it."""
    buf = torch.full((n_bytes + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    buf[n_bytes:] = 0x5A
    return buf, buf[:n_bytes]


def guard_intact(buf):
    return bool((buf[-4096:] == 0x5A).all())


def run_mlp(m, s, work=None):
    d = {k: v.cuda() for k, v in s.items()}
    buf, work = guarded(m.info.work_bytes)
    Y = torch.full_like(d["X"], float("nan"))
    m.mlp(d["X"], d["W1t"], d["W2t"], d["ids"], d["weights"], work, Y)
    st, code = m.check(work)
    assert st == cs.OK, hex(code)
    assert guard_intact(buf)
    return Y


def run_mlp_grad(m, s):
    d = {k: v.cuda() for k, v in s.items()}
    buf, work = guarded(m.info.grad_work_bytes)
    out = {n: torch.full_like(d[n[1:]], float("nan")) for n in ("dX", "dW1t", "dW2t", "dweights")}
    m.mlp_grad(d["X"], d["W1t"], d["W2t"], d["ids"], d["weights"], d["dY"], work, out["dX"], out["dW1t"], out["dW2t"],
               out["dweights"])
    st, code = m.check(work)
    assert st == cs.OK, hex(code)
    assert guard_intact(buf)
    return out


def assert_within(got, ref, bound, what):
    got = f64(got).reshape(ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    worst = float(np.max(np.abs(got - ref) / (bound + TINY))) if ref.size else 0.0
    assert worst <= 1.0, f"{what}: worst error / bound = {worst:.3f}"
