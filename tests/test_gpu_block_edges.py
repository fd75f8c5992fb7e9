"""The routed block on the GPU in rare situations: repeated ids beside infinite weights, infinite norm weights and
gates in rows of every raggedness, slices that start anywhere, and launch variants that need particular sizes.

Bounds as in test_gpu_block.py; where a result is compared with the same call on other inputs, the bits are equal.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import swiglu_mlp_fwd_amd as S  # noqa: E402
import test_gpu_block as G  # noqa: E402
from oracle import block_oracle as B  # noqa: E402
from parity_util import check_guards, guarded  # noqa: E402

DEV = G.DEV


# ----------------------------------------------------------------- experts

def repeated_ids(T, E, k, e, full):
    """The first `full` tokens name e in all k entries and the last token once; every other entry names an expert of its
    own, so that what follows e in the order of the entries is other tokens' experts."""
    others = iter([i for i in range(E) if i != e])
    return np.array([[e if t < full or (t == T - 1 and j == 0) else next(others) for j in range(k)] for t in range(T)],
                    np.int32)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("T,E,k,full,N,K", [
    (8, 60, 8, 1, 72, 4104),     # 9 pairs of one expert, 2 tokens
    (4, 64, 16, 1, 72, 4104),    # 17 pairs, 2 tokens: also more than the 16 columns of the first product
    (16, 64, 4, 2, 72, 4104),    # 9 pairs, 3 tokens
    (32, 64, 2, 8, 136, 4104)])  # 17 pairs, 9 tokens: two passes of tokens in the second product
def test_moe_repeated_ids_of_an_expert_with_non_finite_weights(T, E, k, full, N, K, bad):
    """What the other tokens get does not depend on the weights of an expert that they do not name, however often
    another token names it."""
    e = 3
    x, w = G.normal((T, K), 31, "bf16"), G.normal((T, k), 32, "f32")
    wg, wu = G.normal((E, N, K), 33, "bf16", 0.05), G.normal((E, N, K), 34, "bf16", 0.05)
    wd = G.normal((E, K, N), 35, "bf16", 0.05)
    ids = torch.from_numpy(repeated_ids(T, E, k, e, full)).to(DEV)
    clean = S.moe_fwd(x, wg, wu, wd, ids, w)
    if bad == math.inf:
        want, bound = B.moe_bound(G.host(x), G.host(wg), G.host(wu), G.host(wd), ids.cpu().numpy(), G.host(w), "silu")
        G.within(clean, want, bound, "repeated ids")
    wd[e, ::3] = bad
    y = S.moe_fwd(x, wg, wu, wd, ids, w)
    assert torch.equal(y[full:-1], clean[full:-1])
    named = [*range(full), T - 1]
    assert not torch.isfinite(y[named, ::3]).any()
    keep = torch.arange(K, device=DEV) % 3 != 0
    assert torch.equal(y[:, keep], clean[:, keep])


# ------------------------------------------------------------------- norms

# The last chunk of 8 (bf16) or 4 (fp32) of a ragged row is read from cols - 8 or cols - 4; at -2, -4 and -7 from the
# end lie elements of its own and shared ones.
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [64, 67, 253, 515, 1000, 2051])
@pytest.mark.parametrize("what", ["w_out", "gate"])
def test_norm_infinite_weights_forward(dt, cols, what):
    """One infinite weight or gate: its column of res_out is infinite, so the row's norm gives 0 there and everywhere,
    but for inf * 0 in that column."""
    for back in (2, 4, 7):
        p = G.norm_inputs(5, cols, dt, "norm", True, 1, 7 * cols + back)
        c = cols - back
        p["y"][:, c] = 1.5
        clean, _ = S.block_norm(**p, **G.CONST)
        p[what].view(-1)[c] = math.inf
        ro, z = S.block_norm(**p, **G.CONST)
        others = torch.arange(cols, device=DEV) != c
        assert torch.isinf(ro[:, c]).all() and torch.equal(ro[:, others], clean[:, others]), back
        assert torch.isnan(z[:, c]).all() and (z[:, others] == 0).all(), back


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [64, 67, 515, 2051, 8201])
@pytest.mark.parametrize("what", ["w_out", "gate", "w_in"])
def test_norm_infinite_weights_backward(dt, cols, what):
    """One infinite weight or gate: which elements of dres and dy are NaN, and which infinite, is as the formulas say."""
    for back in (2, 4, 7):
        rows, c = 3, cols - back
        p = G.norm_inputs(rows, cols, dt, "norm", what == "w_in", 0 if what == "w_in" else 1, 9 * cols + back)
        p[what].view(-1)[c] = math.inf
        ro, dro = G.normal((rows, cols), 11, dt), G.normal((rows, cols), 12, dt)
        dz = G.normal((rows, cols), 13, dt) if what == "w_in" else None
        got = S.block_norm_bwd(ro, p["y"], p["w_out"], p["gate"], p["w_in"], dro, dz, **G.CONST)
        with np.errstate(invalid="ignore"):
            want, _ = B.block_norm_bwd(G.host(ro), *(G.host(p[n]) for n in ("y", "w_out", "gate", "w_in")), G.host(dro),
                                       G.host(dz), **G.CONST)
        for name, g, v in zip(("dres", "dy"), got, want):
            g = G.host(g)
            assert np.array_equal(np.isnan(g), np.isnan(v)), f"{name}, {back}: NaN"
            assert np.array_equal(np.isinf(g), np.isinf(v)), f"{name}, {back}: infinite"


# ------------------------------------------------------------------ router

@pytest.mark.parametrize("dt,E", [("bf16", 60), ("bf16", 5), ("f32", 5), ("f32", 130)])
def test_route_takes_slices_that_start_anywhere(dt, E):
    """Contiguous slices whose first element is not on a 16-byte boundary."""
    l, dw = G.normal((9, E), E, dt, 1.5), G.normal((8, 3), 5, "f32")
    part = l[1:]
    assert part.is_contiguous() and part.data_ptr() % 16 != 0
    w, ids = S.route(part, 3)
    want = S.route(part.clone(), 3)
    assert torch.equal(w, want[0]) and torch.equal(ids, want[1])
    assert torch.equal(S.route_bwd(part, ids, dw), S.route_bwd(part.clone(), ids, dw))


# ------------------------------------------------- launch variants and sizes

@pytest.mark.parametrize("spread", ["even", "holes"])
@pytest.mark.parametrize("T,E,k,N,K", [
    (40, 2, 1, 136, 200), (64, 3, 1, 72, 264), (33, 1, 1, 264, 1032),        # up to 64 pairs, over 16 an expert
    (64, 3, 1, 200, 4104), (64, 4, 4, 136, 520),
    (48, 13, 4, 456, 1304), (64, 8, 2, 264, 2056), (30, 4, 2, 520, 712)])     # 32 columns to a workgroup
def test_moe_many_tokens_for_each_expert(T, E, k, N, K, spread):
    G.moe_case(T, E, k, N, K, 800 + T + E, spread=spread)


@pytest.mark.parametrize("T,E,k,N,K", [(1, 8, 2, 136, 256), (8, 8, 2, 72, 4104), (24, 6, 3, 136, 264), (64, 16, 4, 72, 520),
                                       (48, 13, 4, 456, 1304), (40, 2, 1, 264, 1032)])
def test_moe_stays_inside_its_workspace(T, E, k, N, K):
    x, wg, wu, wd, ids, w, y = G.moe_case(T, E, k, N, K, 820 + T)
    ws, yg = guarded((S.moe_workspace_bytes(T, N, K, k),), torch.uint8), guarded((T, K), torch.bfloat16)
    assert torch.equal(S.moe_fwd(x, wg, wu, wd, ids, w, workspace=ws.t, out=yg.t), y)
    check_guards("moe workspace", ws, yg)


@pytest.mark.parametrize("dt,rows,cols,groups", [
    ("bf16", 530, 8201, 1), ("bf16", 530, 8201, 2), ("f32", 530, 4101, 2), ("f32", 530, 8201, 0), ("f32", 530, 8201, 2),
    ("bf16", 600, 2051, 1), ("bf16", 600, 2051, 4), ("f32", 600, 2051, 2), ("bf16", 1540, 4096, 1)])
def test_norm_long_rows_by_several_to_a_workgroup(dt, rows, cols, groups):
    """Forward rows of two chunks to a thread, and backward parts of two or three rows, in an exact workspace."""
    p = G.norm_inputs(rows, cols, dt, "norm", True, groups, rows + cols + groups)
    G.check_norm(p, dt, f"norm {dt} {rows}x{cols} {groups} groups")
    ro, z = S.block_norm(**p, **G.CONST)
    first = S.block_norm_bwd(ro, p["y"], p["w_out"], p["gate"], p["w_in"], z, ro, **G.CONST)
    ws = guarded((S.block_norm_bwd_workspace_bytes(rows, cols, groups),), torch.uint8)
    again = S.block_norm_bwd(ro, p["y"], p["w_out"], p["gate"], p["w_in"], z, ro, **G.CONST, workspace=ws.t)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(first, again))
    check_guards("norm workspace", ws)


@pytest.mark.parametrize("join,pre,groups", [("plain", True, 2), ("plain", False, 1), ("norm", False, 2), ("none", True, 0)])
@pytest.mark.parametrize("dt,cols", [("bf16", 8201), ("f32", 8201), ("f32", 4101)])
def test_norm_long_rows_of_other_forms(dt, cols, join, pre, groups):
    G.check_norm(G.norm_inputs(522, cols, dt, join, pre, groups, cols + groups), dt, f"norm {dt} {join} {pre} {groups} {cols}")
