"""The routed block's oracle against the definitions, closed forms and central differences (CPU)."""
import math

import numpy as np
import pytest

from oracle import block_oracle as B

RNG = np.random.default_rng


def diff(f, v, d, h):
    """Central difference of scalar f at v in direction d."""
    return (f(v + h * d) - f(v - h * d)) / (2 * h)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_matches_differences(score, renorm):
    g = RNG(1)
    l, k = g.normal(size=(6, 11)), 4
    l[2, 3:9] = -np.inf
    dw = g.normal(size=(6, k))
    ids = B.choose(l, k)
    grad, _ = B.route_bwd(l, ids, dw, score, renorm, 2.5)
    d = np.where(l == -np.inf, 0.0, g.normal(size=l.shape))
    num = diff(lambda v: (2.5 * B._q(v, ids, score, renorm) * dw).sum(), l, d, 1e-5)
    # Central differences: error h^2 (third derivative, order 1) + eps / h.
    assert abs((grad * d).sum() - num) < 1e-8
    assert (grad[l == -np.inf] == 0).all()


def test_route_choice_ties_and_masks():
    l = np.array([[1.0, 2.0, 2.0, 0.0], [-np.inf, 5.0, -np.inf, -np.inf], [-np.inf] * 4, [0.0, np.nan, 1.0, 0.0],
                  [np.finfo(np.float32).min] * 4])
    ids = B.choose(l, 3)
    assert ids.tolist() == [[1, 2, 0], [1, -1, -1], [-1, -1, -1], [2, 0, 3], [0, 1, 2]]
    w, _ = B.route(l, 3, "softmax", True, 1.0)
    assert np.allclose(w[0], np.exp([0, 0, -1]) / np.exp([0, 0, -1]).sum())
    assert w[1].tolist() == [1, 0, 0] and w[2].tolist() == [0, 0, 0] and np.isnan(w[3]).all()
    assert np.allclose(w[4], 1 / 3)
    # Sigmoid scores that underflow keep their ratio.
    w, _ = B.route(np.array([[-2000.0, -2001.0]]), 2, "sigmoid", True, 1.0)
    assert np.allclose(w, [[1 / (1 + math.exp(-1)), 1 / (1 + math.exp(1))]])


@pytest.mark.parametrize("join,pre,gates", [("none", True, 0), ("plain", False, 0), ("plain", True, 3), ("norm", False, 1),
                                            ("norm", True, 0), ("norm", True, 3)])
def test_norm_gradients_match_differences(join, pre, gates):
    g = RNG(2)
    rows, cols = 6, 5
    p = dict(res=g.normal(size=(rows, cols)), y=None, w_out=None, gate=None, w_in=None)
    if join != "none":
        p["y"] = g.normal(size=(rows, cols))
    if join == "norm":
        p["w_out"] = g.normal(size=cols)
    if gates:
        p["gate"] = g.normal(size=(gates, cols))
    if pre:
        p["w_in"] = g.normal(size=cols)
    c = dict(skip=0.9, scale=1.5, w_offset=1.0, eps=1e-3)
    dro, dz = g.normal(size=(rows, cols)), g.normal(size=(rows, cols)) if pre else None

    def loss(q):
        ro, z = B.block_norm(**q, **c)
        ro = q["res"] if ro is None else ro
        return (dro * ro).sum() + (0 if z is None else (dz * z).sum())
    ro, _ = B.block_norm(**p, **c)
    ro = p["res"] if ro is None else ro
    grads, terms = B.block_norm_bwd(ro, p["y"], p["w_out"], p["gate"], p["w_in"], dro, dz, **c)
    for name, grad, term in zip(("res", "y", "w_out", "gate", "w_in"), grads, terms):
        if p[name] is None:
            assert grad is None
            continue
        d = g.normal(size=p[name].shape)
        num = diff(lambda v: loss({**p, name: v}), p[name], d, 1e-5)
        assert abs((grad * d).sum() - num) < 1e-7, name
        assert (np.abs(grad) <= term * (1 + 1e-12)).all()


def test_moe_is_the_weighted_sum_of_dense_stages():
    import oracle
    g = RNG(3)
    T, E, N, K = 4, 3, 7, 5
    x, wg, wu, wd = (g.normal(size=s) for s in ((T, K), (E, N, K), (E, N, K), (E, K, N)))
    ids = np.array([[0, 1], [2, -1], [1, 1], [-1, 7]], np.int32)
    w = g.normal(size=(T, 2))
    dense = np.stack([oracle.swiglu_fwd(x, wg[e], wu[e]) @ wd[e].T for e in range(E)])
    want = np.zeros((T, K))
    want[0] = w[0, 0] * dense[0, 0] + w[0, 1] * dense[1, 0]
    want[1] = w[1, 0] * dense[2, 1]
    want[2] = (w[2, 0] + w[2, 1]) * dense[1, 2]
    assert np.allclose(B.moe(x, wg, wu, wd, ids, w, "silu"), want)
    y, bound = B.moe_bound(x, wg, wu, wd, ids, w, "silu")
    assert np.allclose(y, want) and (bound > 0).all()
