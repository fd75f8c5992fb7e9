"""The routed block on the GPU against the fp64 oracle: router, few-token experts, norms around a block.

Bounds (u = 2^-24; a factor 2 of headroom unless stated):
  * router: e^-a is good to a few ulps of its rounded argument, so a score errs by u (16 + a) relative, a = the
    distance of its logit to the greatest one used; a sum of n of them adds n u; scores below the normal range keep
    2^-126 absolute.  The gradient's terms carry the same, and its output rounding.
  * experts: block_oracle.moe_bound.
  * norms: a row sum passes at most 64 additions on its way (a lane's elements, the lanes, the waves), so every term
    errs by (64 + 16) u of its absolute value; sums over rows add one u per row; the second norm turns the error of
    res_out into at most twice its relative size; then the output's rounding.
"""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from parity_util import BF16_HALF_ULP, U32, check_guards, guarded

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import swiglu_mlp_fwd_amd as S  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": BF16_HALF_ULP, "f32": U32}
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def normal(shape, seed, dt, std=1.0):
    a = np.random.default_rng(seed).normal(size=shape) * std
    return torch.from_numpy(a).to(torch.float32).to(DT[dt]).to(DEV)


def host(t):
    return None if t is None else t.double().cpu().numpy()


def within(got, want, bound, what):
    got = host(got)
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN pattern"
    err = np.abs(got - want)[~nan]
    b = np.broadcast_to(bound, want.shape)[~nan]
    assert np.isfinite(err).all(), f"{what}: not finite"
    worst = (err / b).max() if err.size else 0.0
    print(f"{what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


# ------------------------------------------------------------------ router

def route_bounds(l, ids, score, renorm, w):
    """Bound of the weights [T, k]."""
    T, E = l.shape
    live = np.where((ids >= 0), np.take_along_axis(l, np.maximum(ids, 0), 1), 0.0)
    live = np.nan_to_num(live, nan=0.0, posinf=0.0, neginf=0.0)
    far = np.abs(live.max(1, keepdims=True) - live) + np.abs(live)
    return 2 * np.abs(w) * U32 * (16 + far + E) + 2.0 ** -120


def check_route(logits, k, score, renorm, scale, what):
    T, E = logits.shape
    wg, ig = guarded((T, k), torch.float32), guarded((T, k), torch.int32)
    w, ids = S.route(logits, k, score=score, renorm=renorm, scale=scale, out=(wg.t, ig.t))
    check_guards(what, wg, ig)
    l = host(logits)
    want, want_ids = B.route(l, k, score, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids), f"{what}: choice"
    within(w, want, np.nan_to_num(route_bounds(l, want_ids, score, renorm, want), nan=1.0), what)
    # gradient
    dw = normal((T, k), 7, "f32")
    dg = guarded((T, E), logits.dtype)
    d = S.route_bwd(logits, ids, dw, score=score, renorm=renorm, scale=scale, out=dg.t)
    check_guards(what, dg)
    want, terms = B.route_bwd(l, want_ids, host(dw), score, renorm, scale)
    finite = np.where(np.isfinite(l), l, 0.0)
    far = 2 * np.abs(finite).max(1, keepdims=True)
    rnd = ROUND["bf16" if logits.dtype == torch.bfloat16 else "f32"]
    bound = 2 * (terms * 3 * U32 * (16 + far + E) + rnd * np.abs(np.nan_to_num(want))) + 2.0 ** -118
    within(d, want, bound, what + " gradient")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (5, 60, 4), (33, 64, 6), (7, 65, 16), (130, 129, 3), (9, 300, 8),
                                   (3, 512, 1), (4, 1000, 16), (2, 1024, 7), (700, 16, 2), (259, 7, 5)])
def test_route(dt, score, renorm, T, E, k):
    check_route(normal((T, E), T * E + k, dt, 1.5), k, score, renorm, 2.5, f"route {dt} {score} {renorm} {T} {E} {k}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("E", [24, 70, 200])
def test_route_masks_and_special_values(dt, score, renorm, E):
    """Rows: one expert left, none left, all the type's lowest value, all equal, huge spread, tiny scores, a NaN, +inf,
    and masks over most experts."""
    k = 6
    l = normal((24, E), 5, dt, 2.0)
    l[0] = -math.inf
    l[0, E - 2] = 1.0
    l[1] = -math.inf
    l[2] = torch.finfo(l.dtype).min
    l[3] = 0.25
    l[4] = torch.linspace(-90, 80, E)
    l[5] = -200.0 + torch.arange(E) * 0.5
    l[6, 3] = math.nan
    l[7, 5] = math.inf
    l[8] = math.nan
    l[9, ::2] = -math.inf
    l[10, 1:] = -math.inf
    l[11, :E - 3] = -math.inf
    l[12] = -0.0
    l[12, ::3] = 0.0
    check_route(l, k, score, renorm, 1.0, f"route special {dt} {score} {renorm} {E}")


@pytest.mark.parametrize("dt,score,renorm", [("bf16", "softmax", True), ("f32", "softmax", False),
                                             ("bf16", "sigmoid", False), ("f32", "sigmoid", True)])
@pytest.mark.parametrize("E,k", [(3, 2), (5, 5), (8, 8), (9, 3), (16, 16), (31, 8)])
def test_route_many_tokens_few_experts(dt, score, renorm, E, k):
    """Random rows, with masked, equal, lowest-value and NaN rows among them."""
    T = 32771
    l = normal((T, E), 17 * E + k, dt, 2.0)
    l[torch.arange(0, T, 5), torch.arange(0, T, 5) % E] = -math.inf
    l[100::997] = -math.inf
    l[101::997] = 0.25
    l[102::997] = torch.finfo(l.dtype).min
    l[103::997, E - 1] = math.nan
    l[104::997, 0] = math.inf
    l[T - 1] = torch.linspace(-80, 80, E) if E > 1 else 1.0
    check_route(l, k, score, renorm, 1.5, f"route many {dt} {score} {renorm} {E} {k}")


def test_route_equal_logits_take_the_lowest_index():
    g = torch.Generator().manual_seed(3)
    l = torch.randint(0, 4, (300, 96), generator=g).float().to(DEV)
    _, ids = S.route(l, 8)
    assert np.array_equal(ids.cpu().numpy(), B.choose(host(l), 8))
    _, ids = S.route(l.bfloat16(), 16, score="sigmoid")
    assert np.array_equal(ids.cpu().numpy(), B.choose(host(l), 16))


def test_route_bwd_skips_ids_outside_and_adds_repeated_ones():
    l = normal((4, 40), 8, "f32")
    ids = torch.tensor([[3, 3, -1], [40, 2, 1 << 30], [-5, -1, -1], [39, 0, 39]], dtype=torch.int32, device=DEV)
    dw = normal((4, 3), 9, "f32")
    dw[0, 2] = math.nan                          # its id is -1: never read into a result
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = S.route_bwd(l, ids, dw, score=score, renorm=renorm)
            want, terms = B.route_bwd(host(l), ids.cpu().numpy(), np.nan_to_num(host(dw)), score, renorm, 1.0)
            within(d, want, 2 * (terms * 3 * U32 * 80 + U32 * np.abs(want)) + 2.0 ** -118, f"ids {score} {renorm}")


def test_route_offsets_past_32_bits():
    T, E = (1 << 21) + 5, 1024                   # more than 2^31 logits
    l = torch.zeros((T, E), dtype=torch.bfloat16, device=DEV)
    tail = normal((5, E), 11, "bf16")
    l[-5:] = tail
    w, ids = S.route(l, 4)
    want, want_ids = B.route(host(tail), 4, "softmax", True, 1.0)
    assert np.array_equal(ids[-5:].cpu().numpy(), want_ids)
    within(w[-5:], want, route_bounds(host(tail), want_ids, "softmax", True, want), "route tail")
    dw = normal((T, 4), 12, "f32")
    d = S.route_bwd(l, ids, dw)
    want, terms = B.route_bwd(host(tail), want_ids, host(dw[-5:]), "softmax", True, 1.0)
    within(d[-5:], want, 2 * (terms * 3 * U32 * 1100 + BF16_HALF_ULP * np.abs(want)) + 2.0 ** -118, "route tail gradient")
    assert torch.count_nonzero(d[:-5, 4:]).item() == 0
    del l, d
    torch.cuda.empty_cache()


def test_route_layouts_and_empty():
    l = normal((6, 5, 48), 13, "f32")
    w, ids = S.route(l.transpose(0, 1), 3)
    w2, ids2 = S.route(l.transpose(0, 1).contiguous().reshape(30, 48), 3)
    assert w.shape == (5, 6, 3) and torch.equal(w.reshape(30, 3), w2) and torch.equal(ids.reshape(30, 3), ids2)
    w, ids = S.route(l[:0], 3)
    assert w.shape == (0, 5, 3) and ids.shape == (0, 5, 3)
    assert S.route_bwd(l[:0], ids, w).shape == (0, 5, 48)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_router_autograd_matches_differences_of_the_oracle(score, renorm):
    l = normal((8, 32), 14, "f32").requires_grad_(True)
    w, ids = S.router(l, 4, score=score, renorm=renorm, scale=1.5)
    dw = normal((8, 4), 15, "f32")
    (w * dw).sum().backward()
    l64, d = host(l.detach()), np.random.default_rng(16).normal(size=(8, 32))

    def f(v):
        return (1.5 * B._q(v, ids.cpu().numpy(), score, renorm) * host(dw)).sum()
    num = (f(l64 + 1e-5 * d) - f(l64 - 1e-5 * d)) / 2e-5
    # fp32 gradients: u (16 + spread + E) of terms of order 1, 256 of them, beside the difference's own 1e-8.
    assert abs((host(l.grad) * d).sum() - num) < 256 * 3 * U32 * 60


# ------------------------------------------------------------------ experts

def moe_case(T, E, k, N, K, seed, act="silu", spread="even", check=True, what=None):
    x = normal((T, K), seed, "bf16")
    wg, wu = normal((E, N, K), seed + 1, "bf16", 0.05), normal((E, N, K), seed + 2, "bf16", 0.05)
    wd = normal((E, K, N), seed + 3, "bf16", 0.05)
    g = np.random.default_rng(seed + 4)
    if spread == "even":
        ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    elif spread == "skewed":                     # one expert for every token, the others spread
        ids = np.stack([np.concatenate([[E // 2], g.permutation([e for e in range(E) if e != E // 2])[:k - 1]])
                        for _ in range(T)])
    elif spread == "one":                        # every token on one expert, however often it can be named
        ids = np.full((T, k), E - 1)
    else:                                        # holes, and ids outside the experts
        ids = g.integers(-2, E + 2, size=(T, k))
    ids = torch.from_numpy(ids.astype(np.int32)).to(DEV)
    w = normal((T, k), seed + 5, "f32")
    yg = guarded((T, K), torch.bfloat16)
    y = S.moe_fwd(x, wg, wu, wd, ids, w, act=act, out=yg.t)
    what = what or f"moe {T} {E} {k} {N} {K} {act} {spread}"
    check_guards(what, yg)
    want, bound = B.moe_bound(host(x), host(wg), host(wu), host(wd), ids.cpu().numpy(), host(w), act)
    within(y, want, bound, what)
    return x, wg, wu, wd, ids, w, y


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("T,E,k,N,K", [
    (1, 1, 1, 8, 8), (1, 4, 2, 136, 72), (2, 3, 3, 16, 1032), (3, 5, 2, 200, 264), (7, 16, 8, 520, 128),
    (16, 4, 2, 128, 256), (17, 4, 2, 72, 136), (33, 3, 2, 264, 88), (64, 8, 4, 64, 200), (64, 40, 8, 48, 64),
    (5, 13, 3, 1096, 712), (1, 300, 16, 40, 48), (64, 1024, 16, 8, 16)])
def test_moe(act, T, E, k, N, K):
    moe_case(T, E, k, N, K, 100 + T + E, act)


@pytest.mark.parametrize("T,E,k,N,K", [(1, 6, 4, 64, 72), (16, 2, 2, 40, 136), (40, 6, 4, 72, 64), (64, 20, 16, 24, 40)])
def test_moe_repeated_missing_and_foreign_ids(T, E, k, N, K):
    moe_case(T, E, k, N, K, 200 + T, spread="one")
    moe_case(T, E, k, N, K, 300 + T, spread="holes")


@pytest.mark.parametrize("T,E,k,N,K", [(64, 64, 1, 136, 72), (64, 128, 2, 72, 136), (64, 16, 2, 264, 64), (64, 8, 2, 136, 200),
                                       (48, 32, 3, 72, 72), (33, 40, 1, 24, 264), (20, 60, 2, 40, 2608), (64, 70, 1, 40, 1400)])
def test_moe_an_expert_with_far_more_tokens_than_the_others(T, E, k, N, K):
    moe_case(T, E, k, N, K, 250 + T, spread="skewed")


@pytest.mark.parametrize("T,E,k,N,K", [(3, 4, 2, 1000, 2048), (2, 3, 2, 264, 1304), (9, 4, 1, 136, 4104), (5, 7, 3, 5000, 64),
                                       (20, 3, 2, 2056, 520), (40, 2, 2, 136, 3000)])
def test_moe_column_tiles_and_parts(T, E, k, N, K):
    """8 or 16 columns to a workgroup, one part or several, 4 to 16 waves."""
    moe_case(T, E, k, N, K, 270 + T)


def test_moe_no_expert_at_all_and_empty():
    x, wg, wu, wd, ids, w, _ = moe_case(4, 3, 2, 40, 48, 400)
    y = S.moe_fwd(x, wg, wu, wd, torch.full_like(ids, -1), w)
    assert torch.count_nonzero(y).item() == 0
    assert S.moe_fwd(x[:0], wg, wu, wd, ids[:0], w[:0]).shape == (0, 48)
    y = S.moe_fwd(x, wg[:, :0], wu[:, :0], wd[:, :, :0], ids, w)
    assert y.shape == (4, 48) and torch.count_nonzero(y).item() == 0


def test_moe_non_finite_values_stay_with_their_token():
    x, wg, wu, wd, ids, w, y = moe_case(6, 4, 2, 72, 64, 500)
    x2 = x.clone()
    x2[2, 5] = math.nan
    x2[4, 0] = math.inf
    y2 = S.moe_fwd(x2, wg, wu, wd, ids, w)
    assert torch.isnan(y2[2]).all() and not torch.isfinite(y2[4]).any()
    keep = [0, 1, 3, 5]
    assert torch.equal(y2[keep], y[keep])
    w2 = w.clone()
    w2[1, 0] = math.nan
    y2 = S.moe_fwd(x, wg, wu, wd, ids, w2)
    assert torch.isnan(y2[1]).all() and torch.equal(y2[[0, 2, 3, 4, 5]], y[[0, 2, 3, 4, 5]])
    # Weights of experts that no token names are not read.
    lone = torch.zeros_like(ids)
    wg2 = wg.clone()
    wg2[1:] = math.nan
    assert torch.isfinite(S.moe_fwd(x, wg2, wu, wd, lone, w)).all()


def test_moe_stacked_and_distant_experts():
    x, wg, wu, wd, ids, w, y = moe_case(5, 3, 2, 40, 64, 600)
    both = torch.cat([wg, wu], 1)                # [E, 2 N, K]
    y2 = S.moe_fwd(x, both[:, :40], both[:, 40:], wd, ids, w)
    assert torch.equal(y2, y)
    y2 = S.moe_fwd(x, wg.transpose(1, 2).contiguous().transpose(1, 2), wu, wd, ids, w)   # experts not dense
    assert torch.equal(y2, y)
    step = 1 << 30                               # experts 2^30 elements apart: the last starts past 2^31 elements
    far = torch.zeros((2 * step + 3 * 4096,), dtype=torch.bfloat16, device=DEV)
    views = [far.as_strided(t.shape, (step, t.shape[2], 1), 4096 * i) for i, t in enumerate((wg, wu, wd))]
    for v, t in zip(views, (wg, wu, wd)):
        v.copy_(t)
    y2 = S.moe_fwd(x, *views, ids, w)
    assert torch.equal(y2, y)
    del far, views
    torch.cuda.empty_cache()


def test_moe_is_deterministic_and_needs_no_clean_workspace():
    x, wg, wu, wd, ids, w, y = moe_case(24, 6, 3, 136, 264, 700)
    ws = torch.empty(S.moe_workspace_bytes(24, 136, 264, 3), dtype=torch.uint8, device=DEV)
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        for _ in range(2):
            assert torch.equal(S.moe_fwd(x, wg, wu, wd, ids, w, workspace=ws), y)


# ------------------------------------------------------------------ norms

def norm_inputs(rows, cols, dt, join, pre, groups, seed, std=1.0):
    c = lambda s, i, sd=1.0: normal(s, seed + i, dt, sd)
    return dict(res=c((rows, cols), 0, std), y=c((rows, cols), 1, 2 * std) if join != "none" else None,
                w_out=c((cols,), 2) if join == "norm" else None, gate=c((groups, cols), 3) if groups else None,
                w_in=c((cols,), 4) if pre else None)


CONST = dict(skip=0.9, scale=1.5, w_offset=0.5, eps=1e-5)
ROW = 80 * U32                                   # see the header


def check_norm(p, dt, what, const=CONST):
    rows, cols = p["res"].shape
    h = {n: host(v) for n, v in p.items()}
    rnd = ROUND[dt]
    gr = guarded((rows, cols), DT[dt]) if p["y"] is not None else None
    gz = guarded((rows, cols), DT[dt]) if p["w_in"] is not None else None
    ro, z = S.block_norm(**p, **const, out=(gr.t if gr else None, gz.t if gz else None))
    check_guards(what, gr, gz)
    wro, wz = B.block_norm(**h, **const)
    err = np.zeros((rows, cols))
    if wro is not None:
        err = ROW * (np.abs(const["skip"] * h["res"]) + np.abs(wro - const["skip"] * h["res"]))
        within(ro, wro, 2 * (err + rnd * np.abs(wro)) + 1e-37, what + " res_out")
    if wz is not None:
        r = h["res"] if wro is None else wro
        k = 1 / np.sqrt((r * r).mean(1, keepdims=True) + const["eps"])
        w = np.abs(const["w_offset"] + h["w_in"])
        moved = k * w * (err + np.abs(r) * k * np.sqrt((err * err).mean(1, keepdims=True)))
        within(z, wz, 2 * (moved + ROW * np.abs(wz) + rnd * np.abs(wz)) + 1e-37, what + " z")
    # gradients, from the rounded res_out
    ro = p["res"] if ro is None else ro
    dro, dz = normal((rows, cols), 91, dt), normal((rows, cols), 92, dt) if p["w_in"] is not None else None
    outs = [guarded(t.shape, DT[dt]) if t is not None else None
            for t in (p["res"], p["y"], p["w_out"], p["gate"], p["w_in"])]
    got = S.block_norm_bwd(ro, p["y"], w_out=p["w_out"], gate=p["gate"], w_in=p["w_in"], dres_out=dro, dz=dz, **const,
                           out=tuple(None if g is None else g.t for g in outs))
    check_guards(what, *outs)
    want, terms = B.block_norm_bwd(host(ro), h["y"], h["w_out"], h["gate"], h["w_in"], host(dro), host(dz), **const)
    for name, g, v, t, n in zip(("dres", "dy", "dw_out", "dgate", "dw_in"), got, want, terms, (0, 0, rows, rows, rows)):
        if v is None:
            assert g is None
        else:
            # Three products of summed terms at most (both norms and the rows' sum): three times ROW.
            within(g, v, 2 * ((3 * ROW + n * U32) * t + rnd * np.abs(v)) + 1e-37, f"{what} {name}")


JOINS = [("none", True, 0), ("plain", False, 0), ("plain", True, 0), ("plain", False, 1), ("plain", True, 2),
         ("norm", False, 0), ("norm", True, 0), ("norm", False, 2), ("norm", True, 1), ("norm", True, 4)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("join,pre,groups", JOINS)
@pytest.mark.parametrize("rows,cols", [(4, 1), (8, 63), (4, 515), (12, 1000), (8, 2051), (4, 4096), (8, 6001)])
def test_norm(dt, join, pre, groups, rows, cols):
    check_norm(norm_inputs(rows, cols, dt, join, pre, groups, rows * cols), dt,
               f"norm {dt} {join} {pre} {groups} {rows}x{cols}")


@pytest.mark.parametrize("join,pre,groups", JOINS)
@pytest.mark.parametrize("dt,rows,cols", [("bf16", 4, 129), ("bf16", 36, 256), ("bf16", 1036, 251), ("f32", 4, 65),
                                          ("f32", 36, 128), ("f32", 1036, 99)])
def test_norm_half_wave_rows(dt, join, pre, groups, rows, cols):
    check_norm(norm_inputs(rows, cols, dt, join, pre, groups, rows * cols), dt,
               f"norm {dt} {join} {pre} {groups} {rows}x{cols}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,groups", [(1, 8192, 1), (2, 16384, 2), (3, 12289, 0), (1201, 72, 1), (1300, 260, 0),
                                              (2100, 40, 2100), (1800, 136, 600), (1026, 520, 3)])
def test_norm_many_rows_long_rows_many_groups(dt, rows, cols, groups):
    check_norm(norm_inputs(rows, cols, dt, "norm", True, groups, rows + cols), dt,
               f"norm {dt} {rows}x{cols} {groups} groups")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_rows_of_zeros_and_non_finite_rows(dt):
    p = norm_inputs(9, 136, dt, "norm", True, 0, 31)
    p["y"][1] = 0
    p["res"][2] = 0
    p["y"][2] = 0
    check_norm(p, dt, f"norm zero rows {dt}", dict(CONST, eps=1e-20))
    clean = S.block_norm(**p, **CONST)
    p["y"][4, 7] = math.nan
    p["res"][6, 0] = math.inf
    ro, z = S.block_norm(**p, **CONST)
    assert torch.isnan(ro[4]).all() and torch.isnan(z[4]).all() and torch.isinf(ro[6, 0])
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(ro[keep], clean[0][keep]) and torch.equal(z[keep], clean[1][keep])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_unaligned_views_give_the_same(dt):
    """Tensors that start one element into their storage; rows of an odd length."""
    p = norm_inputs(6, 331, dt, "norm", True, 2, 41)
    off = {n: None if v is None else torch.cat([v.new_zeros(1), v.reshape(-1)])[1:].view(v.shape) for n, v in p.items()}
    for a, b in zip(S.block_norm(**p, **CONST), S.block_norm(**off, **CONST)):
        assert torch.equal(a, b)
    d, dz = normal((6, 331), 42, dt), normal((6, 331), 43, dt)
    for a, b in zip(S.block_norm_bwd(p["res"], p["y"], p["w_out"], p["gate"], p["w_in"], d, dz, **CONST),
                    S.block_norm_bwd(off["res"], off["y"], off["w_out"], off["gate"], off["w_in"], d, dz, **CONST)):
        assert torch.equal(a, b)


def test_norm_offsets_past_32_bits():
    rows, cols = (1 << 17) + 2, 16384            # 2^31 + 2^15 elements
    res = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    res[-2:] = normal((2, cols), 51, "bf16")
    w = normal((cols,), 52, "bf16")
    _, z = S.block_norm(res, w_in=w)
    _, want = S.block_norm(res[-2:].clone(), w_in=w)
    assert torch.equal(z[-2:], want) and torch.count_nonzero(z[:-2]).item() == 0
    dz = z                                       # any gradient
    dres, _, _, _, dw = S.block_norm_bwd(res, w_in=w, dz=dz)
    want = S.block_norm_bwd(res[-2:].clone(), w_in=w, dz=dz[-2:].clone())
    assert torch.equal(dres[-2:], want[0]) and torch.count_nonzero(dres[:-2]).item() == 0
    assert torch.equal(dw, want[4])              # zero rows add zeros
    del res, z, dres, dz
    torch.cuda.empty_cache()


def test_norm_empty_rows_and_missing_gradients():
    p = norm_inputs(0, 72, "bf16", "norm", True, 3, 61)
    ro, z = S.block_norm(**p, **CONST)
    assert ro.shape == (0, 72) and z.shape == (0, 72)
    got = S.block_norm_bwd(ro, p["y"], p["w_out"], p["gate"], p["w_in"], ro, z, **CONST)
    assert all(torch.count_nonzero(g).item() == 0 for g in got) and got[3].shape == (3, 72)
    p = norm_inputs(5, 72, "f32", "norm", True, 0, 62)
    ro, z = S.block_norm(**p, **CONST)
    dz = normal((5, 72), 63, "f32")
    a = S.block_norm_bwd(ro, p["y"], p["w_out"], None, p["w_in"], None, dz, **CONST)
    b = S.block_norm_bwd(ro, p["y"], p["w_out"], None, p["w_in"], torch.zeros_like(dz), dz, **CONST)
    assert all(x is None and y is None or torch.equal(x, y) for x, y in zip(a, b))


def test_norm_gradients_are_deterministic():
    p = norm_inputs(1500, 520, "bf16", "norm", True, 2, 71)
    ro, z = S.block_norm(**p, **CONST)
    first = S.block_norm_bwd(ro, p["y"], p["w_out"], p["gate"], p["w_in"], z, ro, **CONST)
    ws = torch.full((S.block_norm_bwd_workspace_bytes(1500, 520, 2),), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        again = S.block_norm_bwd(ro, p["y"], p["w_out"], p["gate"], p["w_in"], z, ro, **CONST, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_norm_autograd_matches_differences_of_the_oracle():
    p = {n: v.requires_grad_(True) for n, v in norm_inputs(8, 40, "f32", "norm", True, 2, 81).items()}
    dro, dz = normal((8, 40), 82, "f32"), normal((8, 40), 83, "f32")
    ro, z = S.block_norms(p["res"], p["y"], p["w_out"], p["gate"], p["w_in"], **CONST)
    ((ro * dro).sum() + (z * dz).sum()).backward()
    h = {n: host(v.detach()) for n, v in p.items()}
    for i, name in enumerate(p):
        d = np.random.default_rng(84 + i).normal(size=h[name].shape)

        def f(s):
            a, b = B.block_norm(**{**h, name: h[name] + s * d}, **CONST)
            return (a * host(dro)).sum() + (b * host(dz)).sum()
        num = (f(1e-5) - f(-1e-5)) / 2e-5
        # Terms of order 10 at most, 320 of them, each within 3 ROW; the difference's own error is below 1e-7.
        assert abs((host(p[name].grad) * d).sum() - num) < 320 * 10 * 3 * ROW, name


# ------------------------------------------------------------------ together

def block_step(p):
    ro, z = S.block_norm(p["res"], p["y"], w_out=p["w_out"], w_in=p["w_in"])
    w, ids = S.route(z.float() @ p["wr"], 2)
    return ro, z, w, ids, S.moe_fwd(z, p["wg"], p["wu"], p["wd"], ids, w)


def block_params(seed):
    n = norm_inputs(6, 264, "bf16", "norm", True, 0, seed)
    n.update(wr=normal((264, 5), seed + 10, "f32"), wg=normal((5, 72, 264), seed + 11, "bf16", 0.05),
             wu=normal((5, 72, 264), seed + 12, "bf16", 0.05), wd=normal((5, 264, 72), seed + 13, "bf16", 0.05))
    return n


def test_block_on_another_stream():
    p = block_params(900)
    want = block_step(p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = block_step(p)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_block_replays_in_a_graph():
    p = block_params(910)
    n = norm_inputs(64, 264, "bf16", "norm", True, 2, 911)
    d = normal((64, 264), 912, "bf16")
    logits, dw = normal((40, 24), 913, "f32"), normal((40, 4), 914, "f32")
    ids0 = S.route(logits, 4)[1]
    logits5 = normal((6, 5), 915, "f32")

    def step():
        ro, z = S.block_norm(p["res"], p["y"], w_out=p["w_out"], w_in=p["w_in"])
        w, ids = S.route(logits5, 2)
        y = S.moe_fwd(z, p["wg"], p["wu"], p["wd"], ids, w)
        g = S.block_norm_bwd(n["res"], n["y"], n["w_out"], n["gate"], n["w_in"], d, d, **CONST)
        return (ro, z, w, ids, y, *g, S.route_bwd(logits, ids0, dw))
    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for rep in range(4):
        for t in captured:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, eager)):
            assert torch.equal(a, b), f"replay {rep}, output {i}"
        step()                                   # eager work between the replays
        torch.cuda.synchronize()


def test_example_runs():
    spec = importlib.util.spec_from_file_location("routed_block", os.path.join(ROOT, "examples", "routed_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    first, last = ex.train(steps=12, tokens=96, width=128, hidden=192, experts=6, topk=2)
    assert last < 0.8 * first
    y = ex.decode(steps=3, batch=4, blocks=2, width=128, hidden=192, experts=6, topk=2)
    assert y.shape == (4, 128) and torch.isfinite(y.float()).all()
