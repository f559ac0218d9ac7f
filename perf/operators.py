"""Workloads of the mixture-of-experts operators, for timing and comparison.

Five operators, as one expert layer of a transformer uses them: the router (scores, top-k,
weights), its gradient, the dispatch plan (which expert's rows each assignment takes), the
experts' MLP of every token (two products per chosen expert, combined by weight) and its
backward pass.  With ``own`` false, ``run`` computes them from elementary torch operations
in 32 bits (64 where selection compares near-equal scores); with ``own`` true it calls this
package.
"""

import math

import numpy as np
import torch

own = False

PLAN_ROWS = 128  # an expert's rows start at a multiple of this in the dispatch order


# ------------------------------------------------------------------ cases


def _route(op, T, E, k, score, groups, group_limit, group_top, bias, renorm, scale, f32, masked, **more):
    return dict(op=op, T=T, E=E, k=k, score=score, groups=groups, group_limit=group_limit, group_top=group_top,
                bias=bias, renorm=renorm, scale=scale, f32=f32, masked=masked, **more)


def _mlp(op, T, E, k, D, N1, act, **more):
    return dict(op=op, T=T, E=E, k=k, D=D, N1=N1, act=act, **more)


def listed():
    return [
        # one token's routing in a serving loop: launch latency is all there is
        _route("route", 1, 64, 8, "softmax", 1, 1, 1, False, True, 1.0, False, False, name="route_token"),
        # a long prompt with balance biases and groups: 8 of 256 experts out of 4 of 8 groups
        _route("route", 32768, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5, True, False, name="route_prompt"),
        # ragged batch, odd expert count, some experts switched off for some tokens
        _route("route", 1777, 60, 4, "softmax", 1, 1, 1, False, False, 1.0, True, True, name="route_ragged"),
        # gradients of the router's scores: a small ragged batch and a training batch
        _route("route_grad", 777, 60, 4, "softmax", 1, 1, 1, False, False, 1.0, False, False, name="route_grad_ragged"),
        _route("route_grad", 32768, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5, True, False, name="route_grad_batch"),
        # dispatch plan of a decoding batch and of a training batch
        dict(op="plan", T=64, E=64, k=8, dropped=0.0, name="plan_decode"),
        dict(op="plan", T=32768, E=256, k=8, dropped=0.1, name="plan_batch"),
        # one token in decoding: 8 experts' weights are read for a single row
        _mlp("mlp", 1, 64, 8, 2048, 1024, "swiglu", name="mlp_token"),
        # a decoding batch: every expert's weights, few rows each
        _mlp("mlp", 48, 64, 8, 2048, 1024, "swiglu", name="mlp_decode"),
        # a prompt or training forward
        _mlp("mlp", 4096, 64, 8, 2048, 1024, "swiglu", name="mlp_prompt"),
        # backward: a small ragged GeLU layer, and a training batch
        _mlp("mlp_grad", 333, 17, 2, 1000, 776, "gelu", name="mlp_grad_ragged"),
        _mlp("mlp_grad", 4096, 64, 8, 2048, 1024, "swiglu", name="mlp_grad_batch"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "plan", "mlp", "mlp", "mlp_grad"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(4, 32)
        limit = rng.randint(1, groups)
        k = rng.randint(1, min(8, limit * (E // groups)))
        score, renorm = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6
        if op == "route_grad" and renorm:
            k = max(k, 2)  # a single renormalised weight is constant: its gradient is zero
        return _route(op, _log(rng, 1, 32768), E, k, score, groups, limit, rng.choice([1, 2]), rng.random() < 0.5,
                      renorm, rng.choice([1.0, 2.5]), rng.random() < 0.5, op == "route" and rng.random() < 0.2)
    if op == "plan":
        return dict(op=op, T=_log(rng, 1, 32768), E=rng.randint(2, 256), k=rng.randint(1, 8),
                    dropped=rng.choice([0.0, 0.1]))
    T, E, k = _log(rng, 1, 4096), rng.randint(4, 96), rng.randint(1, 4)
    D, N1 = 8 * _log(rng, 16, 400), 8 * _log(rng, 16, 200)
    while E * D * N1 > 64 * 2048 * 1024:
        E = max(4, E // 2)
        D = max(128, D // 16 * 8)
    while T * k * D * N1 > 4096 * 8 * 2048 * 1024:
        T = T // 2
    return _mlp(op, T, E, min(k, E), D, N1, rng.choice(["swiglu", "gelu"]))


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _topk_ids(g, T, E, k):
    """Expert choices with some experts more popular than others, best first."""
    logits = _randn(g, T, E) + 0.7 * _randn(g, E)
    return torch.argsort(logits, dim=1, descending=True)[:, :k].to(torch.int32).contiguous(), logits


def prepare(case, seed):
    g, c = _gen(seed), case
    T, E, k = c["T"], c["E"], c["k"]
    s = {"case": c}
    if c["op"] in ("route", "route_grad"):
        logits = 1.5 * _randn(g, T, E) + 0.5 * _randn(g, E)
        if c["masked"]:
            # experts switched off for a token (-inf), and a few tokens that may use none
            off = torch.rand((T, E), generator=g, device="cuda") < 0.3
            off |= (torch.arange(T, device="cuda") % 97 == 5)[:, None]
            logits = logits.masked_fill(off, float("-inf"))
        s["logits"] = logits if c["f32"] else logits.to(torch.bfloat16)
        s["bias"] = 0.1 * _randn(g, E) if c["bias"] else None
        if c["op"] == "route_grad":
            s["ids"] = _select(s["logits"], s["bias"], c)[0]
            s["dweights"] = _randn(g, T, k)
    elif c["op"] == "plan":
        s["ids"], _ = _topk_ids(g, T, E, k)
        if c["dropped"]:
            s["ids"].masked_fill_(torch.rand((T, k), generator=g, device="cuda") < c["dropped"], -1)
    else:
        D, N1, G = c["D"], c["N1"], 2 if c["act"] == "swiglu" else 1
        s["X"] = _randn(g, T, D).to(torch.bfloat16)
        s["W1t"] = torch.empty((E, G * N1, D), dtype=torch.bfloat16, device="cuda").normal_(0, D ** -0.5, generator=g)
        s["W2t"] = torch.empty((E, D, N1), dtype=torch.bfloat16, device="cuda").normal_(0, N1 ** -0.5, generator=g)
        s["ids"], logits = _topk_ids(g, T, E, k)
        s["weights"] = torch.softmax(logits.gather(1, s["ids"].long()), dim=1).contiguous()
        if c["op"] == "mlp_grad":
            s["dY"] = _randn(g, T, D).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms


def _select(logits, bias, c):
    """(ids, scores of the ids, scores) in 64 bits: the order of near-equal scores counts."""
    T, E = logits.shape
    l = logits.double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        ex = torch.exp(l - torch.amax(l, dim=1, keepdim=True))
        score = ex / ex.sum(dim=1, keepdim=True)
    off = l == float("-inf")
    key = score if bias is None else score + bias.double()
    key = key.masked_fill(off, float("-inf"))
    G = c["groups"]
    if G > 1:
        kg = key.view(T, G, E // G)
        best = torch.sort(kg, dim=2, descending=True).values[:, :, : c["group_top"]].sum(dim=2)
        order = torch.argsort(best, dim=1, descending=True, stable=True)[:, : c["group_limit"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter(1, order, True)
        key = kg.masked_fill(~keep[:, :, None], float("-inf")).view(T, E)
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, : c["k"]]
    none = key.gather(1, order) == float("-inf")
    return order.masked_fill(none, -1).to(torch.int32), score.gather(1, order).masked_fill(none, 0.0), score


def _route_plain(s):
    c = s["case"]
    ids, picked, _ = _select(s["logits"], s["bias"], c)
    total = picked.sum(dim=1, keepdim=True)
    w = torch.where(total > 0, picked / total, picked) if c["renorm"] else picked
    return {"ids": ids, "weights": (c["scale"] * w).float()}


def _route_grad_plain(s):
    c = s["case"]
    l = s["logits"].float()
    ids, dw = s["ids"].long(), s["dweights"].float() * c["scale"]
    dense = torch.zeros_like(l).scatter(1, ids, dw)           # gradient of the normalised weights
    chosen = torch.zeros_like(l).scatter(1, ids, 1.0)
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        ex = torch.exp(l - torch.amax(l, dim=1, keepdim=True))
        score = ex / ex.sum(dim=1, keepdim=True)
    if c["renorm"]:
        total = (score * chosen).sum(dim=1, keepdim=True)
        inner = (dense * score).sum(dim=1, keepdim=True) / total
        dscore = chosen * (dense - inner) / total
    else:
        dscore = dense
    if c["score"] == "sigmoid":
        d = dscore * score * (1.0 - score)
    else:
        d = score * (dscore - (dscore * score).sum(dim=1, keepdim=True))
    return {"dlogits": d.to(s["logits"].dtype)}


def _plan_slots(T, E, k):
    return -(-(T * k + (PLAN_ROWS - 1) * min(E, T * k)) // PLAN_ROWS) * PLAN_ROWS


def _plan_plain(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    A, S = T * k, _plan_slots(T, E, k)
    flat = s["ids"].reshape(A).long()
    e = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device).index_add_(0, e, torch.ones_like(e))
    starts = torch.cumsum(counts, 0) - counts
    padded = (counts[:E] + PLAN_ROWS - 1) // PLAN_ROWS * PLAN_ROWS
    offsets = torch.cat([torch.zeros_like(padded[:1]), torch.cumsum(padded, 0)])
    order = torch.argsort(e, stable=True)
    eo = e[order]
    slot = torch.where(eo < E, offsets[eo] + torch.arange(A, device=e.device) - starts[eo], torch.full_like(eo, S))
    row_of = torch.full((S + 1,), -1, dtype=torch.int64, device=e.device).scatter(0, slot, order)[:S]
    slot_of = torch.empty_like(slot).scatter(0, order, torch.where(slot < S, slot, torch.full_like(slot, -1)))
    return {"counts": counts[:E].int(), "offsets": offsets.int(), "slot_of": slot_of.int().view(T, k),
            "row_of": row_of.int()}


def _grouped(s):
    """Rows of X by expert, padded to the largest expert: (rows index [E, cap], valid, place of
    each assignment in the flattened [E * cap])."""
    c = s["case"]
    A, E = c["T"] * c["k"], c["E"]
    e = s["ids"].reshape(A).long()
    counts = torch.bincount(e, minlength=E)
    cap = int(counts.max())
    order = torch.argsort(e, stable=True)
    starts = torch.cumsum(counts, 0) - counts
    place = torch.empty_like(order).scatter(0, order, e[order] * cap + torch.arange(A, device=e.device) - starts[e[order]])
    rows = torch.zeros(E * cap, dtype=torch.int64, device=e.device).scatter(0, place, torch.arange(A, device=e.device))
    valid = torch.zeros(E * cap, dtype=torch.float32, device=e.device).scatter(0, place, 1.0)
    return rows, valid.view(E, cap, 1), place, cap


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


_GELU_C = math.sqrt(2.0 / math.pi)


def _mlp_plain(s):
    c = s["case"]
    T, E, k, D, N1 = c["T"], c["E"], c["k"], c["D"], c["N1"]
    rows, valid, place, cap = _grouped(s)
    x = s["X"].float()[rows // k].view(E, cap, D)
    z = torch.bmm(x, s["W1t"].float().transpose(1, 2))
    if c["act"] == "swiglu":
        g = z[:, :, :N1]
        h = g * _sigmoid(g) * z[:, :, N1:]
    else:
        h = z * _sigmoid(2.0 * _GELU_C * (z + 0.044715 * z * z * z))
    o = torch.bmm(h, s["W2t"].float().transpose(1, 2)).view(E * cap, D)
    y = (o[place].view(T, k, D) * s["weights"][:, :, None]).sum(dim=1)
    return {"Y": y.to(torch.bfloat16)}


def _mlp_grad_plain(s):
    c = s["case"]
    T, E, k, D, N1 = c["T"], c["E"], c["k"], c["D"], c["N1"]
    rows, valid, place, cap = _grouped(s)
    W1, W2 = s["W1t"].float(), s["W2t"].float()
    x = s["X"].float()[rows // k].view(E, cap, D) * valid
    dy = s["dY"].float()[rows // k].view(E, cap, D) * valid
    w = s["weights"].reshape(-1)[rows].view(E, cap, 1)
    z = torch.bmm(x, W1.transpose(1, 2))
    dh = torch.bmm(dy, W2)
    if c["act"] == "swiglu":
        g, u = z[:, :, :N1], z[:, :, N1:]
        sg = _sigmoid(g)
        h = g * sg * u
        dhw = dh * w
        dz = torch.cat([dhw * u * sg * (1.0 + g * (1.0 - sg)), dhw * g * sg], dim=2)
    else:
        sg = _sigmoid(2.0 * _GELU_C * (z + 0.044715 * z * z * z))
        h = z * sg
        dz = dh * w * (sg + z * sg * (1.0 - sg) * 2.0 * _GELU_C * (1.0 + 3.0 * 0.044715 * z * z))
    dweights = (dh * h).sum(dim=2).view(E * cap)[place].view(T, k)
    dW2 = torch.bmm(dy.transpose(1, 2), h * w)
    dW1 = torch.bmm(dz.transpose(1, 2), x)
    dx = torch.bmm(dz, W1).view(E * cap, D)[place].view(T, k, D).sum(dim=1)
    bf = torch.bfloat16
    return {"dX": dx.to(bf), "dW1t": dW1.to(bf), "dW2t": dW2.to(bf), "dweights": dweights}


# ------------------------------------------------------------------ the framework's calls


def _handle(s):
    """The layer object and the buffers that a user's program keeps beside it."""
    import tile_level_sync_gb300 as cs

    c = s["case"]
    T, E, k, dev = c["T"], c["E"], c["k"], "cuda"
    if c["op"] in ("route", "route_grad"):
        m = cs.Moe(cs.make_moe_desc(T=T, experts=E, top_k=k, score=c["score"], groups=c["groups"],
                                    group_limit=c["group_limit"], group_top=c["group_top"], renorm=c["renorm"],
                                    scale=c["scale"], logits_f32=c["f32"]))
        out = {"ids": torch.empty((T, k), dtype=torch.int32, device=dev),
               "weights": torch.empty((T, k), dtype=torch.float32, device=dev)}
        if c["op"] == "route_grad":
            out = {"dlogits": torch.empty_like(s["logits"])}
        return m, out, None
    if c["op"] == "plan":
        m = cs.Moe(cs.make_moe_desc(T=T, experts=E, top_k=k))
        plan = torch.empty(m.info.plan_bytes // 4, dtype=torch.int32, device=dev)
        return m, m.plan_views(plan), plan
    m = cs.Moe(cs.make_moe_desc(T=T, D=c["D"], N1=c["N1"], experts=E, top_k=k, act=c["act"]))
    if c["op"] == "mlp":
        return m, {"Y": torch.empty_like(s["X"])}, torch.empty(m.info.work_bytes, dtype=torch.uint8, device=dev)
    out = {"dX": torch.empty_like(s["X"]), "dW1t": torch.empty_like(s["W1t"]), "dW2t": torch.empty_like(s["W2t"]),
           "dweights": torch.empty_like(s["weights"])}
    return m, out, torch.empty(m.info.grad_work_bytes, dtype=torch.uint8, device=dev)


def _run_own(s):
    if "kept" not in s:
        s["kept"] = _handle(s)
    m, out, work = s["kept"]
    op = s["case"]["op"]
    if op == "route":
        m.route(s["logits"], s["bias"], out["ids"], out["weights"])
    elif op == "route_grad":
        m.route_grad(s["logits"], s["ids"], s["dweights"], out["dlogits"])
    elif op == "plan":
        m.plan(s["ids"], work)
    elif op == "mlp":
        m.mlp(s["X"], s["W1t"], s["W2t"], s["ids"], s["weights"], work, out["Y"])
    else:
        m.mlp_grad(s["X"], s["W1t"], s["W2t"], s["ids"], s["weights"], s["dY"], work, out["dX"], out["dW1t"],
                   out["dW2t"], out["dweights"])
    return out


_PLAIN = {"route": _route_plain, "route_grad": _route_grad_plain, "plan": _plan_plain, "mlp": _mlp_plain,
          "mlp_grad": _mlp_grad_plain}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work


def work(case):
    c = case
    T, E, k = c["T"], c["E"], c["k"]
    A = T * k
    if c["op"] == "route":
        return {"bytes": T * E * (4 if c["f32"] else 2) + 8 * A + (4 * E if c["bias"] else 0), "flops": 4 * T * E}
    if c["op"] == "route_grad":
        return {"bytes": 2 * T * E * (4 if c["f32"] else 2) + 8 * A, "flops": 8 * T * E}
    if c["op"] == "plan":
        return {"bytes": 8 * A + 4 * _plan_slots(T, E, k) + 8 * E, "flops": 2 * A}
    D, N1, G = c["D"], c["N1"], 2 if c["act"] == "swiglu" else 1
    active = E * (1.0 - (1.0 - k / E) ** T)        # experts that some token chooses, if all are as likely
    weights = active * (G + 1) * N1 * D * 2
    if c["op"] == "mlp":
        return {"bytes": weights + 2 * T * D * 2 + 8 * A, "flops": 2 * A * (G + 1) * N1 * D}
    # recomputes the hidden layer (G products), then its gradient (1), the inputs' (G), the weights' (G + 1)
    grads = E * (G + 1) * N1 * D * 2
    return {"bytes": weights + grads + 3 * T * D * 2 + 12 * A, "flops": 2 * A * (3 * G + 2) * N1 * D}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_scores(l, score):
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.exp(-np.logaddexp(0.0, -l))
        return np.exp(l - np.logaddexp.reduce(l, axis=1, keepdims=True))


def _exact_route(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].double().cpu().numpy()
    score = np.nan_to_num(_exact_scores(l, c["score"]))
    key = score + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    key[np.isneginf(l)] = -np.inf
    if c["groups"] > 1:
        kg = key.reshape(T, c["groups"], -1)
        top = -np.sort(-kg, axis=2)[:, :, : c["group_top"]].sum(axis=2)
        drop = np.argsort(-top, axis=1, kind="stable")[:, c["group_limit"]:]
        kg[np.arange(T)[:, None], drop] = -np.inf
        key = kg.reshape(T, E)
    pick = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.where(np.isneginf(np.take_along_axis(key, pick, 1)), 0.0, np.take_along_axis(score, pick, 1))
    if c["renorm"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return {"ids": None, "weights": c["scale"] * w}


def _exact_route_grad(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].double().cpu().numpy()
    ids = s["ids"].cpu().numpy()
    dw = s["dweights"].double().cpu().numpy() * c["scale"]
    p = _exact_scores(l, c["score"])
    ps = np.take_along_axis(p, ids, 1)
    total = ps.sum(axis=1, keepdims=True)
    ds = (dw - (dw * ps).sum(axis=1, keepdims=True) / total) / total if c["renorm"] else dw
    d = np.zeros((T, E))
    if c["score"] == "sigmoid":
        np.put_along_axis(d, ids, ds * ps * (1.0 - ps), 1)
    else:
        np.put_along_axis(d, ids, ds, 1)
        d = p * (d - (ds * ps).sum(axis=1, keepdims=True))
    return {"dlogits": d}


def _exact_mlp(c, s):
    T, E, k, D, N1 = c["T"], c["E"], c["k"], c["D"], c["N1"]
    grad = c["op"] == "mlp_grad"
    x, ids = s["X"].double(), s["ids"].long()
    w = s["weights"].double()
    dev = x.device
    y = torch.zeros((T, D), dtype=torch.float64, device=dev)
    if grad:
        dy = s["dY"].double()
        dW1, dW2 = torch.zeros(s["W1t"].shape, dtype=torch.float64, device=dev), torch.zeros(
            s["W2t"].shape, dtype=torch.float64, device=dev)
        dwt = torch.zeros((T, k), dtype=torch.float64, device=dev)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        a, b = s["W1t"][e].double(), s["W2t"][e].double()
        z = x[t] @ a.T
        if c["act"] == "swiglu":
            gate, up = z[:, :N1], z[:, N1:]
            sig = torch.sigmoid(gate)
            h = gate * sig * up
        else:
            th = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            h = 0.5 * z * (1 + th)
        ww = w[t, j][:, None]
        if not grad:
            y.index_add_(0, t, ww * (h @ b.T))
            continue
        dh = dy[t] @ b
        dwt[t, j] = (dh * h).sum(dim=1)
        dhw = dh * ww
        if c["act"] == "swiglu":
            dz = torch.cat([dhw * up * (sig + gate * sig * (1 - sig)), dhw * gate * sig], dim=1)
        else:
            inner = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
            dz = dhw * (0.5 * (1 + th) + 0.5 * z * (1 - th ** 2) * inner)
        dW1[e], dW2[e] = dz.T @ x[t], dy[t].T @ (ww * h)
        y.index_add_(0, t, dz @ a)
    return {"dX": y, "dW1t": dW1, "dW2t": dW2, "dweights": dwt} if grad else {"Y": y}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "plan":
        return None
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "route_grad":
        return _exact_route_grad(c, s)
    return _exact_mlp(c, s)
