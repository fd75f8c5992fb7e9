"""fp64 reference of the routed block over any number of tokens: the order of rows, the products grouped by expert, the
sum of a token's rows, their gradients, and the clipping of gradients.

Plain numpy from the definitions; it shares no code with the HIP path.  The products also return error bounds, from
sums of absolute values (the caller names the unit roundoff of the output type).
"""
from __future__ import annotations

import math

import numpy as np

from .swiglu_oracle import ACTIVATION_GRADS, ACTIVATIONS

U32 = 2.0 ** -24


def plan(ids, E):
    """(offsets, src, pos) of pairs ids [T, k]: by expert, then by pair; dropped ones last, as complements."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.array(sorted(range(len(key)), key=lambda p: (key[p], p)), np.int64)
    offsets = np.array([(key < e).sum() for e in range(E + 1)], np.int64)
    src = np.array([p if key[p] < E else ~p for p in order], np.int64)
    pos = np.empty(len(key), np.int64)
    for r, p in enumerate(order):
        pos[p] = r if key[p] < E else ~r
    return offsets, src, pos.reshape(np.shape(ids))


def gather(x, src, k):
    rows = np.zeros((len(src), x.shape[1]))
    for r, p in enumerate(src):
        if p >= 0:
            rows[r] = x[p // k]
    return rows


def combine(rows, pos, weights=None):
    """(y, sums of absolute terms)."""
    T, k = pos.shape
    w = np.ones((T, k)) if weights is None else weights
    y, a = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                y[t] += w[t, j] * rows[pos[t, j]]
                a[t] += np.abs(w[t, j] * rows[pos[t, j]])
    return y, a


def combine_bwd(dy, rows, pos, weights=None):
    """(drows, dweights, sums of absolute terms of dweights)."""
    T, k = pos.shape
    w = np.ones((T, k)) if weights is None else weights
    drows, dw, a = np.zeros_like(rows), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = pos[t, j]
            if r >= 0:
                drows[r] = w[t, j] * dy[t]
                dw[t, j] = (dy[t] * rows[r]).sum()
                a[t, j] = np.abs(dy[t] * rows[r]).sum()
    return drows, dw, a


def _runs(offsets, R):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1) if offsets[e + 1] > offsets[e]]


def _gamma(n):
    return (n + 1) * U32 / (1 - (n + 1) * U32)


def mm(x, w, offsets, rnd):
    """(y, bound) of y[r] = x[r] W_e^T, rounded once to a type of unit roundoff rnd."""
    R, (_, N, K) = x.shape[0], w.shape
    y, b = np.zeros((R, N)), np.zeros((R, N))
    for e, i, j in _runs(offsets, R):
        y[i:j] = x[i:j] @ w[e].T
        b[i:j] = _gamma(K) * (np.abs(x[i:j]) @ np.abs(w[e]).T)
    return y, 2 * (b + rnd * np.abs(y))


def mm_bwd(x, w, dy, offsets, rnd, edy=None):
    """((dx, bound), (dw, bound)); edy: errors that dy already has."""
    R, (E, N, K) = x.shape[0], w.shape
    edy = np.zeros_like(dy) if edy is None else edy
    dx, bx = np.zeros((R, K)), np.zeros((R, K))
    dw, bw = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e, i, j in _runs(offsets, R):
        dx[i:j] = dy[i:j] @ w[e]
        bx[i:j] = (_gamma(N) * np.abs(dy[i:j]) + edy[i:j]) @ np.abs(w[e])
        dw[e] = dy[i:j].T @ x[i:j]
        bw[e] = (_gamma(j - i) * np.abs(dy[i:j]) + edy[i:j]).T @ np.abs(x[i:j])
    return (dx, 2 * (bx + rnd * np.abs(dx))), (dw, 2 * (bw + rnd * np.abs(dw)))


def gate_up(x, wg, wu, offsets, act, rnd):
    """(h, bound) of h = act(g) u.  |act'| < 1.2; the activation itself errs by 1e-5 of its value where the result is
    rounded to 8 bits and by 16 fp32 ulps otherwise."""
    R, (_, N, K) = x.shape[0], wg.shape
    h, b = np.zeros((R, N)), np.zeros((R, N))
    own = 1e-5 if rnd > 1e-3 else 16 * U32
    for e, i, j in _runs(offsets, R):
        g, u = x[i:j] @ wg[e].T, x[i:j] @ wu[e].T
        eg, eu = (_gamma(K) * (np.abs(x[i:j]) @ np.abs(w[e]).T) for w in (wg, wu))
        a = ACTIVATIONS[act](g)
        h[i:j] = a * u
        b[i:j] = 1.2 * eg * (np.abs(u) + eu) + np.abs(a) * eu + (own + rnd) * np.abs(h[i:j])
    return h, 2 * b


def gate_up_bwd(x, wg, wu, dh, offsets, act, rnd):
    """((dx, bound), (dwg, bound), (dwu, bound)).  dg and du are rounded to the type of unit roundoff rnd, so each errs
    by rnd of its value besides what its factors carry (|act'| < 1.2, |act''| < 1.2)."""
    R, (E, N, K) = x.shape[0], wg.shape
    dg, du = np.zeros((R, N)), np.zeros((R, N))
    eg_, eu_ = np.zeros((R, N)), np.zeros((R, N))
    own = 2e-5 if rnd > 1e-3 else 32 * U32
    for e, i, j in _runs(offsets, R):
        g, u = x[i:j] @ wg[e].T, x[i:j] @ wu[e].T
        eg, eu = (_gamma(K) * (np.abs(x[i:j]) @ np.abs(w[e]).T) for w in (wg, wu))
        a, da, d = ACTIVATIONS[act](g), ACTIVATION_GRADS[act](g), dh[i:j]
        dg[i:j], du[i:j] = d * u * da, d * a
        eg_[i:j] = np.abs(d) * (eu * 1.2 + np.abs(u) * (1.2 * eg + own)) + rnd * np.abs(dg[i:j])
        eu_[i:j] = np.abs(d) * (1.2 * eg + own * (np.abs(a) + np.abs(g))) + rnd * np.abs(du[i:j])
    (xg, bg), (wgg, bwg) = mm_bwd(x, wg, dg, offsets, 0.0, eg_)
    (xu, bu), (wuu, bwu) = mm_bwd(x, wu, du, offsets, 0.0, eu_)
    # dx is one sum of 2 N terms.
    extra = _gamma(2 * N) - _gamma(N)
    for e, i, j in _runs(offsets, R):
        bg[i:j] += 2 * extra * (np.abs(dg[i:j]) @ np.abs(wg[e]) + np.abs(du[i:j]) @ np.abs(wu[e]))
    dx = xg + xu
    return ((dx, bg + bu + 2 * rnd * np.abs(dx)), (wgg, bwg + 2 * rnd * np.abs(wgg)),
            (wuu, bwu + 2 * rnd * np.abs(wuu)))


def clip(grads, max_norm, eps=1e-6):
    """(norm, factor) of fp64 arrays."""
    norm = math.sqrt(sum(float((g * g).sum()) for g in grads))
    f = max_norm / (norm + eps)
    return norm, (1.0 if f > 1.0 else f)
