"""fp64 reference of the routed block: router, routed MLP, norms around a block.

Plain numpy from the definitions; it shares no code with the HIP path.  Where
an error bound needs them, a function also returns the sums of absolute
values its result is made of.
"""
from __future__ import annotations

import numpy as np

from .swiglu_oracle import ACTIVATIONS


def choose(logits, k):
    """ids [T, k]: the greatest logits, equal ones in order of index; -1 where only -inf (or NaN) is left."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(l, order, 1) == -np.inf, -1, order).astype(np.int32)


def poisoned(logits, score):
    """Tokens whose weights are NaN."""
    bad = np.isnan(logits).any(1)
    if score == "softmax":
        bad |= (logits == np.inf).any(1)
    return bad


def _log_scores(l, score):
    """log of the scores up to a term that a row shares (softmax)."""
    if score == "softmax":
        return l
    return -np.logaddexp(0.0, -l)


def _q(l, ids, score, renorm):
    """Weights of ids before scale [T, k] (0 for ids outside the experts or masked), for finite or -inf logits."""
    T, E = l.shape
    q = np.zeros(ids.shape)
    for t in range(T):
        live = [j for j, e in enumerate(ids[t]) if 0 <= e < E and l[t, e] != -np.inf]
        if not live:
            continue
        ls = _log_scores(l[t, ids[t, live]], score)
        if renorm or score == "softmax":         # from the greatest: log sums of huge values lose the sum
            over = ls if renorm else l[t]
            top = over.max()
            q[t, live] = np.exp(ls - top) / np.exp(over - top).sum()
        else:
            q[t, live] = np.exp(ls)
    return q


def route(logits, k, score, renorm, scale):
    l = np.asarray(logits, np.float64)
    ids = choose(l, k)
    bad = poisoned(l, score)
    w = np.full(ids.shape, np.nan)
    w[~bad] = scale * _q(l[~bad], ids[~bad], score, renorm)
    return w, ids


def route_bwd(logits, ids, dweights, score, renorm, scale):
    """(dlogits, the absolute terms of each)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    out, terms = np.zeros((T, E)), np.zeros((T, E))
    bad = poisoned(l, score)
    for t in range(T):
        if bad[t]:
            out[t] = np.nan
            continue
        q = _q(l[t:t + 1], ids[t:t + 1], score, renorm)[0]
        live = [j for j, e in enumerate(ids[t]) if 0 <= e < E and l[t, e] != -np.inf]
        d = np.zeros(len(q))
        d[live] = scale * dweights[t][live]
        m, ma = (q * d).sum(), np.abs(q * d).sum()
        if score == "softmax" and not renorm:
            top = l[t].max()
            if top == -np.inf:
                continue
            p = np.exp(l[t] - top)
            p /= p.sum()
            de, da = np.zeros(E), np.zeros(E)
            for j in live:
                de[ids[t, j]] += d[j]
                da[ids[t, j]] += abs(d[j])
            out[t], terms[t] = p * (de - m), p * (da + ma)
            continue
        for j in live:
            e = ids[t, j]
            c = 1.0 if score == "softmax" else 1.0 / (1.0 + np.exp(min(l[t, e], 700.0)))
            if renorm:
                g, ga = q[j] * (d[j] - m) * c, q[j] * (abs(d[j]) + ma) * c
            else:
                g, ga = d[j] * q[j] * c, abs(d[j]) * q[j] * c
            out[t, e] += g
            terms[t, e] += ga
    return out, terms


def moe(x, wg, wu, wd, ids, weights, act):
    """y [T, K] of the routed MLP; wg, wu [E, N, K], wd [E, K, N] may be dicts {expert: array}."""
    E = len(wg)
    y = np.zeros_like(x, dtype=np.float64)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if 0 <= e < E:
                h = ACTIVATIONS[act](wg[e] @ x[t]) * (wu[e] @ x[t])
                y[t] += weights[t, j] * (wd[e] @ h)
    return y


def moe_bound(x, wg, wu, wd, ids, weights, act, u=2.0 ** -24, out=2.0 ** -8):
    """(y, elementwise error bound): fp32 accumulation of the first products (gamma of K + 1 terms), the activation
    (8 ulps), h kept to 16 bits (2^-16), fp32 accumulation of the second (its operands are split in two: gamma of
    2 N + k + 1 terms), the output's rounding; with a factor 2."""
    E = len(wg)
    T, K = x.shape
    y = moe(x, wg, wu, wd, ids, weights, act)
    err = np.zeros((T, K))

    def gamma(n):
        return n * u / (1 - n * u)
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E:
                continue
            g, v = wg[e] @ x[t], wu[e] @ x[t]
            G = gamma(K + 1)
            eg, ev = G * (np.abs(wg[e]) @ np.abs(x[t])), G * (np.abs(wu[e]) @ np.abs(x[t]))
            a = ACTIVATIONS[act](g)
            h = a * v
            eh = 1.2 * np.abs(v) * eg + np.abs(a) * ev + eg * ev + (8 * u + 2.0 ** -16) * np.abs(h)
            n = 2 * h.shape[0] + ids.shape[1] + 1
            err[t] += abs(weights[t, j]) * (np.abs(wd[e]) @ (eh + gamma(n) * (np.abs(h) + eh)))
    return y, 2 * (err + out * np.abs(y)) + 1e-30


def _rms(v, eps):
    k = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v * k, k


def _gate_rows(gate, rows):
    return 1.0 if gate is None else np.repeat(gate, rows // gate.shape[0], axis=0)


def block_norm(res, y, w_out, gate, w_in, skip, scale, w_offset, eps):
    """(res_out or None, z or None)."""
    r, ro, z = np.asarray(res, np.float64), None, None
    if y is not None:
        n = y if w_out is None else _rms(y, eps)[0] * (w_offset + w_out)
        r = ro = skip * r + scale * _gate_rows(gate, r.shape[0]) * n
    if w_in is not None:
        z = _rms(r, eps)[0] * (w_offset + w_in)
    return ro, z


def block_norm_bwd(res_out, y, w_out, gate, w_in, dres_out, dz, skip, scale, w_offset, eps):
    """((dres, dy, dw_out, dgate, dw_in), the same sums with every term's absolute value)."""
    rows, cols = (dz if dz is not None else dres_out).shape
    t = np.zeros((rows, cols)) if dres_out is None else np.asarray(dres_out, np.float64)
    ta = np.abs(t)
    dw_in = dw_in_a = dy = dya = dw_out = dw_out_a = dgate = dgate_a = None

    def rms_t(v, d, da):
        h, k = _rms(v, eps)
        ha = np.abs(h)
        return (k * (d - h * (d * h).mean(1, keepdims=True)),
                k * (da + ha * (da * ha).mean(1, keepdims=True)))
    if w_in is not None:
        h, _ = _rms(res_out, eps)
        dw_in, dw_in_a = (dz * h).sum(0), np.abs(dz * h).sum(0)
        w = w_offset + w_in
        d, da = rms_t(res_out, dz * w, np.abs(dz * w))
        t, ta = t + d, ta + da
    if y is None:
        return (t, None, None, None, dw_in), (ta, None, None, None, dw_in_a)
    G = _gate_rows(gate, rows)
    h = y if w_out is None else _rms(y, eps)[0]
    w = 1.0 if w_out is None else w_offset + w_out
    if gate is not None:
        v = scale * t * h * w
        va = np.abs(scale) * ta * np.abs(h * w)
        shape = (gate.shape[0], rows // gate.shape[0], cols)
        dgate, dgate_a = v.reshape(shape).sum(1), va.reshape(shape).sum(1)
    d, da = scale * t * G, np.abs(scale) * ta * np.abs(G)
    if w_out is None:
        dy, dya = d, da
    else:
        dw_out, dw_out_a = (d * h).sum(0), (da * np.abs(h)).sum(0)
        dy, dya = rms_t(y, d * w, da * np.abs(w))
    return ((skip * t, dy, dw_out, dgate, dw_in),
            (np.abs(skip) * ta, dya, dw_out_a, dgate_a, dw_in_a))
