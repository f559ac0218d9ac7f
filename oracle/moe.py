"""Plain fp64 definitions of the mixture-of-experts layer: the router and its gradient, the
dispatch order, the experts' MLP and its gradients, token by token and assignment by
assignment, with a bound on what 16-bit stores and fp32 sums may change in each result.

The bounds count, for every value: half a bf16 step (2^-8 of the value) where the device
stores it in bf16, half an fp16 step (2^-11 of the largest of its 32 neighbours at most)
where it stores a slot's row of the output before the sum over a token's experts, one fp32 step (2^-23) of the sum of magnitudes for every term of an fp32
sum, and 2^-20 of the value for the device's exponential and division; each error is
carried through the formula that uses the value by that formula's largest slope.
"""

import numpy as np

BF16 = 2.0 ** -8
HALF = 2.0 ** -11  # an fp16 step of a value of the largest size in its block of 32, at most
STEP = 2.0 ** -23
FAST = 2.0 ** -20
TILE_ROWS = 128


def sigmoid(x):
    return np.exp(-np.logaddexp(0.0, -x))


def _below(l, most):
    """l - most, 0 where both are +inf."""
    with np.errstate(invalid="ignore"):
        return np.where(l == most, 0.0, l - most)


def scores(logits, kind):
    """fp64 scores; a logit of -inf or NaN scores 0, one of +inf what it tends to (softmax: all there
    is, shared with other +inf)."""
    l = np.where(np.isnan(logits), -np.inf, logits)
    with np.errstate(invalid="ignore"):
        if kind == "sigmoid":
            return sigmoid(l)
        m = l.max(axis=1, keepdims=True)
        e = np.where(np.isneginf(l), 0.0, np.exp(_below(l, np.where(np.isneginf(m), 0.0, m))))
        total = e.sum(axis=1, keepdims=True)
        return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route(logits, bias, top_k, kind="softmax", groups=1, group_limit=0, group_top=1, renorm=False, scale=1.0):
    """(ids, weights), by sorting python tuples: no vectorised selection to get wrong.  Where no bias
    and no sum of two keys decides, experts go by their logits: scores that 64 bits round to the
    same number grow with them all the same."""
    T, E = logits.shape
    s = scores(logits, kind)
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k))
    size = E // groups
    limit = group_limit or groups
    for t in range(T):
        key = [(-np.inf if np.isneginf(logits[t, e]) or np.isnan(logits[t, e])
                else s[t, e] + (0.0 if bias is None else float(bias[e]))) for e in range(E)]
        key = [-np.inf if np.isnan(x) else x for x in key]  # a bias of NaN
        if bias is None and (groups == 1 or group_top == 1):
            key = [-np.inf if np.isnan(x) else x for x in logits[t].astype(np.float64)]
        rank = []
        for g in range(groups):
            best = sorted(key[g * size:(g + 1) * size], reverse=True)[:group_top]
            # a group without as many keys as its rank adds up is last, beside a key of +inf too
            rank.append((np.inf if -np.inf in best else -sum(best), g))
        kept = {g for _, g in sorted(rank)[:limit]}
        order = sorted((-key[e], e) for e in range(E) if e // size in kept and key[e] > -np.inf)[:top_k]
        for j, (_, e) in enumerate(order):
            ids[t, j], weights[t, j] = e, s[t, e]
        if renorm and order:
            chosen = ids[t, :len(order)]
            l = logits[t, chosen].astype(np.float64)
            ls = l if kind == "softmax" else -np.logaddexp(0.0, -l)
            w = np.exp(_below(ls, ls.max()))
            weights[t, :len(order)] = w / w.sum()
    return ids, scale * weights


def route_weights(logits, ids, kind, renorm, scale):
    """The weights as a function of the logits for fixed ids (what the gradient is of)."""
    s = scores(logits, kind)
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if renorm:
        w = w / w.sum(axis=1, keepdims=True)
    return scale * w


def route_grad(logits, ids, dweights, kind, renorm, scale):
    """dlogits through the scores' Jacobian, one token at a time."""
    T, E = logits.shape
    s = scores(logits, kind)
    out = np.zeros((T, E))
    for t in range(T):
        on = ids[t] >= 0
        c = ids[t, on]
        if not len(c):
            continue
        w = s[t, c]
        jw = np.eye(len(c)) * scale                       # d weight_j / d score_c(i)
        if renorm:
            total = w.sum()
            jw = scale * (np.eye(len(c)) / total - np.outer(w, np.ones(len(c))) / total ** 2)
        ds = np.zeros(E)
        np.add.at(ds, c, dweights[t, on] @ jw)
        if kind == "sigmoid":
            out[t] = ds * s[t] * (1.0 - s[t])
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
    return out


def slots(T, E, top_k):
    A = T * top_k
    return -(-(A + (TILE_ROWS - 1) * min(E, A)) // TILE_ROWS) * TILE_ROWS


def plan(ids, E):
    """The dispatch order by appending assignments to their experts' lists."""
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for a, e in enumerate(ids.reshape(-1)):
        if 0 <= e < E:
            lists[e].append(a)
    offsets, at = [0], 0
    row_of = np.full(slots(T, E, k), -1, np.int32)
    slot_of = np.full(T * k, -1, np.int32)
    for rows in lists:
        for i, a in enumerate(rows):
            row_of[at + i], slot_of[a] = a, at + i
        at += -(-len(rows) // TILE_ROWS) * TILE_ROWS
        offsets.append(at)
    return {"counts": np.array([len(r) for r in lists], np.int32), "offsets": np.array(offsets, np.int32),
            "slot_of": slot_of.reshape(T, k), "row_of": row_of}


def _blocks_of_32(o):
    """The largest magnitude of each row's block of 32 columns, at every column."""
    n, d = o.shape
    pad = np.zeros((n, -(-d // 32) * 32))
    pad[:, :d] = np.abs(o)
    return np.repeat(pad.reshape(n, -1, 32).max(axis=2), 32, axis=1)[:, :d]


_C = np.sqrt(2.0 / np.pi)


def _hidden(x, w1, act, dz):
    """h, its fp32 error bound for an error of dz in the pre-activations, and what the
    backward pass needs: slopes of h by gate (or z) and by up, with their error bounds."""
    z = x @ w1.T
    if act == "swiglu":
        n = z.shape[1] // 2
        g, u, dg, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
        s = sigmoid(g)
        h = g * s * u
        err = 1.1 * np.abs(u) * dg + np.abs(g * s) * du + 1.1 * dg * du + FAST * np.abs(h)
        slope_g, slope_u = u * (s + g * s * (1 - s)), g * s
        # |silu'| <= 1.1, |silu''| <= 0.5; the slope's terms carry the fast sigmoid's error
        e_g = 1.1 * du + 0.5 * np.abs(u) * dg + FAST * np.abs(u) * (s + np.abs(g) * s * (2 - s))
        e_u = 1.1 * dg + FAST * np.abs(slope_u)
        return h, err, [(slope_g, e_g), (slope_u, e_u)]
    t = np.tanh(_C * (z + 0.044715 * z ** 3))
    h = 0.5 * z * (1 + t)
    # |gelu'| <= 1.13; the sigmoid's argument carries a few fp32 steps of its own size
    arg = 2 * _C * np.abs(z + 0.044715 * z ** 3)
    fast = FAST + 4 * STEP * arg * (1 - t ** 2)
    err = 1.13 * dz + fast * np.abs(z)
    slope = 0.5 * (1 + t) + 0.5 * z * (1 - t ** 2) * _C * (1 + 3 * 0.044715 * z ** 2)
    return h, err, [(slope, 1.2 * dz + fast * (1 + np.abs(z) * 2 * _C * (1 + 3 * 0.044715 * z ** 2)))]


def mlp(X, W1t, W2t, ids, weights, act):
    """(Y, bound)."""
    T, D = X.shape
    E, N1 = W2t.shape[0], W2t.shape[2]
    Y, bound = np.zeros((T, D)), np.zeros((T, D))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        x = X[t]
        dz = D * STEP * (np.abs(x) @ np.abs(W1t[e]).T)
        h, dh, _ = _hidden(x, W1t[e], act, dz)
        dh = dh + BF16 * (np.abs(h) + dh)
        w = weights[t, j][:, None]
        o = h @ W2t[e].T
        np.add.at(Y, t, w * o)
        a2 = np.abs(W2t[e]).T
        np.add.at(bound, t, np.abs(w) * HALF * (_blocks_of_32(o) * (1 + BF16)))
        np.add.at(bound, t, np.abs(w) * (dh @ a2 + (N1 + ids.shape[1] + 4) * STEP * (np.abs(h) @ a2)))
    return Y, bound + BF16 * (np.abs(Y) + bound)


def mlp_grad(X, W1t, W2t, ids, weights, dY, act):
    """{name: (gradient, bound)}."""
    T, D = X.shape
    E, _, N1 = W2t.shape
    dX, bX = np.zeros((T, D)), np.zeros((T, D))
    dW1, b1 = np.zeros(W1t.shape), np.zeros(W1t.shape)
    dW2, b2 = np.zeros(W2t.shape), np.zeros(W2t.shape)
    dw, bw = np.zeros(ids.shape), np.zeros(ids.shape)
    for e in range(E):
        t, j = np.nonzero(ids == e)
        n = len(t)
        if not n:
            continue
        x, y, a, b = X[t], dY[t], W1t[e], W2t[e]
        w = weights[t, j][:, None]
        ez = D * STEP * (np.abs(x) @ np.abs(a).T)
        h, eh, slopes = _hidden(x, a, act, ez)
        dh = y @ b
        edh = D * STEP * (np.abs(y) @ np.abs(b))
        dw[t, j] = (dh * h).sum(axis=1)
        bw[t, j] = (edh * (np.abs(h) + eh) + np.abs(dh) * eh + (N1 + 8) * STEP * np.abs(dh * h)).sum(axis=1)
        dz = np.concatenate([w * dh * s for s, _ in slopes], axis=1)
        ez = np.concatenate([np.abs(w) * (edh * (np.abs(s) + es) + np.abs(dh) * es) + FAST * np.abs(w * dh * s)
                             for s, es in slopes], axis=1)
        ez = ez + BF16 * (np.abs(dz) + ez)
        np.add.at(dX, t, dz @ a)
        np.add.at(bX, t, HALF * _blocks_of_32(dz @ a) * (1 + BF16))
        np.add.at(bX, t, ez @ np.abs(a) + (a.shape[0] + ids.shape[1]) * STEP * (np.abs(dz) @ np.abs(a)))
        dW1[e] = dz.T @ x
        b1[e] = ez.T @ np.abs(x) + (n + 64) * STEP * (np.abs(dz).T @ np.abs(x))
        wh = w * h
        ewh = np.abs(w) * eh
        ewh = ewh + BF16 * (np.abs(wh) + ewh)
        dW2[e] = y.T @ wh
        b2[e] = np.abs(y).T @ ewh + (n + 64) * STEP * (np.abs(y).T @ np.abs(wh))
    return {"dX": (dX, bX + BF16 * (np.abs(dX) + bX)), "dW1t": (dW1, b1 + BF16 * (np.abs(dW1) + b1)),
            "dW2t": (dW2, b2 + BF16 * (np.abs(dW2) + b2)), "dweights": (dw, bw)}
