"""The oracle of rows in order of expert against the definitions and central differences (CPU)."""
import math

import numpy as np
import pytest

from oracle import group_oracle as G

RNG = np.random.default_rng


def test_plan_is_a_permutation_in_order():
    ids = np.array([[2, 0], [-1, 2], [5, 1], [0, 2]])
    offsets, src, pos = G.plan(ids, 4)
    assert offsets.tolist() == [0, 2, 3, 6, 6]
    assert src.tolist() == [1, 6, 5, 0, 3, 7, ~2, ~4]
    assert pos.tolist() == [[3, 0], [~6, 4], [~7, 2], [1, 5]]


def problem(seed=0, T=5, k=2, E=3, N=4, K=6):
    g = RNG(seed)
    ids = g.integers(-1, E, size=(T, k))
    offsets, src, pos = G.plan(ids, E)
    x = g.normal(size=(T, K))
    wg, wu, wd = g.normal(size=(E, N, K)), g.normal(size=(E, N, K)), g.normal(size=(E, K, N))
    w = g.uniform(0.1, 1.0, size=(T, k))
    return dict(ids=ids, offsets=offsets, src=src, pos=pos, x=x, wg=wg, wu=wu, wd=wd, w=w, dy=g.normal(size=(T, K)), k=k)


def forward(p, act):
    xr = G.gather(p["x"], p["src"], p["k"])
    h, _ = G.gate_up(xr, p["wg"], p["wu"], p["offsets"], act, 0.0)
    rows, _ = G.mm(h, p["wd"], p["offsets"], 0.0)
    return G.combine(rows, p["pos"], p["w"])[0], xr, h, rows


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_routed_mlp_matches_the_definition_token_by_token(act):
    p = problem()
    y, *_ = forward(p, act)
    for t in range(5):
        want = np.zeros(6)
        for j in range(2):
            e = p["ids"][t, j]
            if e >= 0:
                h = G.ACTIVATIONS[act](p["wg"][e] @ p["x"][t]) * (p["wu"][e] @ p["x"][t])
                want += p["w"][t, j] * (p["wd"][e] @ h)
        assert np.allclose(y[t], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_match_differences(act):
    p = problem(3)
    y, xr, h, rows = forward(p, act)
    drows, dw, _ = G.combine_bwd(p["dy"], rows, p["pos"], p["w"])
    (dh, _), (dwd, _) = G.mm_bwd(h, p["wd"], drows, p["offsets"], 0.0)
    (dxr, _), (dwg, _), (dwu, _) = G.gate_up_bwd(xr, p["wg"], p["wu"], dh, p["offsets"], act, 0.0)
    dx, _ = G.combine(dxr, p["pos"])
    grads = dict(x=dx, w=dw, wg=dwg, wu=dwu, wd=dwd)
    for name, grad in grads.items():
        d = RNG(9).normal(size=grad.shape)

        def loss(s):
            q = dict(p)
            q[name] = p[name] + s * d
            return (forward(q, act)[0] * p["dy"]).sum()
        # Central differences: error h^2 (third derivative) + eps / h; values of the order of 100.
        num = (loss(1e-5) - loss(-1e-5)) / 2e-5
        assert abs((grad * d).sum() - num) < 1e-6 * max(1.0, abs(num)), name


def test_clip_factor():
    g = [np.array([3.0]), np.array([[4.0]])]
    assert G.clip(g, 10.0) == (5.0, 1.0)
    n, f = G.clip(g, 1.0, 0.0)
    assert n == 5.0 and f == 0.2
    assert math.isnan(G.clip([np.array([np.nan])], 1.0)[1])
