"""The routed block's entry points without a GPU: refusals of the C ABI and of the wrappers, workspace sizes."""
import math

import pytest
import torch

import swiglu_mlp_fwd_amd as S
import swiglu_mlp_fwd_amd.block_ops as ops
from test_abi_host import A, EALIGN, EARG, EDTYPE, ENULL, ESHAPE, EUNSUP, EWS, L, MIS, OK  # noqa: F401


def test_route_validation(L):  # noqa: F811
    f = L.swiglu_route_fwd
    assert f(2, 0, 0, 4, 8, 2, A, 1.0, A, A, None) == EARG             # score
    assert f(0, 0, 2, 4, 8, 2, A, 1.0, A, A, None) == EDTYPE
    assert f(0, 0, 0, -1, 8, 2, A, 1.0, A, A, None) == ESHAPE
    assert f(0, 0, 0, 1 << 31, 8, 2, A, 1.0, A, A, None) == ESHAPE
    for E, k in ((0, 1), (1025, 1), (8, 0), (8, 9), (64, 17)):
        assert f(0, 0, 0, 4, E, k, A, 1.0, A, A, None) == ESHAPE
    assert f(0, 0, 0, (1 << 27) + 1, 8, 2, A, 1.0, A, A, None) == EUNSUP
    for s in (math.nan, math.inf, -math.inf):
        assert f(0, 0, 0, 4, 8, 2, A, s, A, A, None) == EARG
    assert f(0, 0, 0, 4, 8, 2, None, 1.0, A, A, None) == ENULL
    assert f(0, 0, 0, 4, 8, 2, A, 1.0, None, A, None) == ENULL
    assert f(0, 0, 0, 4, 8, 2, A, 1.0, A, None, None) == ENULL
    assert f(0, 0, 0, 4, 8, 2, MIS, 1.0, A, A, None) == EALIGN
    assert f(0, 0, 0, 4, 8, 2, A, 1.0, A + 2, A, None) == EALIGN
    assert f(1, 1, 1, 0, 8, 2, None, 1.0, None, None, None) == OK
    b = L.swiglu_route_bwd
    assert b(2, 0, 0, 4, 8, 2, A, 1.0, A, A, A, None) == EARG
    assert b(0, 0, 0, 4, 8, 9, A, 1.0, A, A, A, None) == ESHAPE
    assert b(0, 0, 0, 4, 8, 2, A, 1.0, A, A, None, None) == ENULL
    assert b(0, 0, 0, 4, 8, 2, A, 1.0, A, A, MIS, None) == EALIGN
    assert b(0, 0, 0, 4, 8, 2, A, 1.0, None, A, A, None) == ENULL
    assert b(0, 0, 0, 0, 8, 2, None, 1.0, None, None, None, None) == OK


def test_moe_validation(L):  # noqa: F811
    f = L.swiglu_moe_fwd
    T, E, k, N, K = 4, 8, 2, 40, 64
    need = L.swiglu_moe_workspace_bytes(T, N, K, k)
    # The hidden activations in two bf16 parts; y in 128 parts (2 column tiles of 32 for 256 CUs).
    assert need == T * k * N * 4 + 128 * T * K * 4
    assert L.swiglu_moe_workspace_bytes(T, N, 8192, k) == T * k * N * 4

    def call(act=0, T=T, E=E, k=k, N=N, K=K, x=A, ids=A, w=A, wg=A, sg=N * K, wu=A, su=N * K, wd=A, sd=N * K, y=A, ws=A,
             n=1 << 40):
        return f(act, T, E, k, N, K, x, ids, w, wg, sg, wu, su, wd, sd, y, ws, n, None)
    assert call(act=2) == EARG
    for bad in (dict(T=-1), dict(T=65), dict(N=-8), dict(N=44), dict(K=60), dict(E=0), dict(E=1025), dict(k=0), dict(k=9),
                dict(E=64, k=17), dict(sg=N * K - 8), dict(su=N * K + 4), dict(sd=-8), dict(sd=0), dict(su=1 << 50)):
        assert call(**bad) == ESHAPE, bad
    assert call(N=(1 << 20) + 8, sg=1 << 40, su=1 << 40, sd=1 << 40) == EUNSUP
    assert L.swiglu_moe_workspace_bytes(65, N, K, k) == 0 and L.swiglu_moe_workspace_bytes(4, 44, K, k) == 0
    for name in ("x", "ids", "w", "wg", "wu", "wd", "y"):
        assert call(**{name: None}) == ENULL, name
        assert call(**{name: A + 2}) == EALIGN, name
    assert call(ws=None) == EWS and call(ws=A + 16) == EALIGN and call(n=need - 1) == EWS
    assert call(T=0, x=None, ids=None, w=None, wg=None, wu=None, wd=None, y=None, ws=None) == OK
    assert call(K=0, x=None, y=None) == OK


def test_norm_validation(L):  # noqa: F811
    f, b = L.swiglu_block_norm_fwd, L.swiglu_block_norm_bwd
    rows, cols = 6, 33

    def fwd(dt=0, rows=rows, cols=cols, groups=2, res=A, y=A, wo=A, gate=A, wi=A, skip=1.0, scale=1.0, off=0.0, eps=1e-6,
            ro=A, z=A):
        return f(dt, rows, cols, groups, res, y, wo, gate, wi, skip, scale, off, eps, ro, z, None)
    assert fwd(dt=2) == EDTYPE
    for bad in (dict(rows=-1), dict(cols=0), dict(groups=-1), dict(groups=4), dict(rows=1 << 31)):
        assert fwd(**bad) == ESHAPE, bad
    assert fwd(cols=16385) == EUNSUP and fwd(rows=1 << 27) == EUNSUP and fwd(rows=1 << 21, groups=1 << 21) == EUNSUP
    for bad in (dict(skip=math.nan), dict(scale=math.inf), dict(off=math.nan), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=math.inf), dict(groups=0), dict(gate=None), dict(y=None), dict(wi=None), dict(ro=A, y=None, wo=None,
                                                                                                   gate=None, groups=0)):
        assert fwd(**bad) == EARG, bad
    assert fwd(y=None, wo=None, gate=None, groups=0, wi=None, ro=None, z=None) == EARG
    for name in ("res", "ro", "z"):
        assert fwd(**{name: None}) == ENULL, name
    for name in ("res", "y", "wo", "gate", "wi", "ro", "z"):
        assert fwd(**{name: A + 2}) == EALIGN, name
    assert fwd(rows=0, res=None, ro=None, z=None) == OK

    need = L.swiglu_block_norm_bwd_workspace_bytes(rows, cols, 2)
    assert need > 0 and need % 256 == 0
    assert L.swiglu_block_norm_bwd_workspace_bytes(rows, cols, 4) == 0
    assert L.swiglu_block_norm_bwd_workspace_bytes(rows, 16385, 2) == 0

    def bwd(dt=0, rows=rows, cols=cols, groups=2, ro=A, y=A, wo=A, gate=A, wi=A, dro=A, dz=A, eps=1e-6, dres=A, dy=A,
            dwo=A, dgate=A, dwi=A, ws=A, n=1 << 40):
        return b(dt, rows, cols, groups, ro, y, wo, gate, wi, dro, dz, 1.0, 1.0, 0.0, eps, dres, dy, dwo, dgate, dwi, ws, n,
                 None)
    assert bwd(dt=9) == EDTYPE and bwd(cols=0) == ESHAPE and bwd(eps=0.0) == EARG and bwd(groups=3, rows=7) == ESHAPE
    for name in ("ro", "dz", "dres", "dy", "dwo", "dgate", "dwi"):
        assert bwd(**{name: None}) == ENULL, name
    for name in ("y", "wo", "gate", "wi"):
        assert bwd(**{name: None}) == EARG, name
    for name in ("ro", "y", "wo", "gate", "wi", "dro", "dz", "dres", "dy", "dwo", "dgate", "dwi"):
        assert bwd(**{name: A + 2}) == EALIGN, name
    assert bwd(ws=None) == EWS and bwd(n=need - 1) == EWS and bwd(ws=A + 16) == EALIGN


# ----------------------------------------------------------------- wrappers

@pytest.fixture
def no_library(monkeypatch):
    def fail():
        raise AssertionError("the library was reached by a call that should have been rejected")
    monkeypatch.setattr(ops, "lib", fail)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


GPU_ONLY = "GPU tensors only"


def test_route_wrapper(no_library):
    for k in (0, 9, 17):
        with pytest.raises(ValueError, match="k must"):
            ops.route(f32(4, 8), k)
    with pytest.raises(ValueError, match="experts"):
        ops.route(f32(4, 1025), 1)
    with pytest.raises(ValueError, match="score"):
        ops.route(f32(4, 8), 2, score="tanh")
    with pytest.raises(TypeError):
        ops.route(f32(4, 8).half(), 2)
    for out in ((f32(4, 3), i32(4, 2)), (f32(4, 2), f32(4, 2)), (None, i32(4, 2)), (f32(2, 4).t(), i32(4, 2))):
        with pytest.raises((ValueError, TypeError)):
            ops.route(f32(4, 8), 2, out=out)
    with pytest.raises(ValueError, match=GPU_ONLY):
        ops.route(bf(2, 2, 8), 2)
    for ids, dw in ((i32(4, 2), f32(4, 3)), (i32(3, 2), f32(3, 2))):
        with pytest.raises(ValueError):
            ops.route_bwd(f32(4, 8), ids, dw)
    with pytest.raises(TypeError):
        ops.route_bwd(f32(4, 8), i32(4, 2).long(), f32(4, 2))
    with pytest.raises(TypeError):
        ops.route_bwd(f32(4, 8), i32(4, 2), f32(4, 2), out=bf(4, 8))
    with pytest.raises(ValueError, match=GPU_ONLY):
        ops.route_bwd(f32(4, 8), i32(4, 2), f32(4, 2))


def test_moe_wrapper(no_library):
    good = dict(x=bf(4, 64), wg=bf(8, 40, 64), wu=bf(8, 40, 64), wd=bf(8, 64, 40), ids=i32(4, 2), weights=f32(4, 2))
    for name, bad, exc in (("x", f32(4, 64), TypeError), ("wu", bf(8, 48, 64), ValueError), ("wd", bf(8, 40, 64), ValueError),
                           ("wg", bf(40, 64), ValueError), ("wg", bf(8, 40, 72), ValueError), ("ids", i32(3, 2), ValueError),
                           ("ids", i32(4, 2).long(), TypeError), ("weights", f32(4, 3), ValueError),
                           ("weights", bf(4, 2), TypeError)):
        with pytest.raises(exc):
            ops.moe_fwd(**{**good, name: bad})
    with pytest.raises(ValueError, match="64 tokens"):
        ops.moe_fwd(**{**good, "x": bf(65, 64), "ids": i32(65, 2), "weights": f32(65, 2)})
    for out in (bf(4, 72), f32(4, 64)):
        with pytest.raises((ValueError, TypeError)):
            ops.moe_fwd(**good, out=out)
    with pytest.raises(ValueError, match="workspace"):
        ops.moe_fwd(**good, workspace=torch.zeros(64, 64, dtype=torch.uint8).t())
    with pytest.raises(ValueError, match=GPU_ONLY):
        ops.moe_fwd(**good)


def test_norm_wrapper(no_library):
    r = f32(6, 40)
    for kw in (dict(), dict(w_out=f32(40), w_in=f32(40)), dict(gate=f32(40), w_in=f32(40)), dict(y=f32(6, 41)),
               dict(y=r, w_out=f32(41)), dict(y=r, w_in=f32(1, 40)), dict(y=r, gate=f32(4, 40)), dict(y=r, gate=f32(0, 40)),
               dict(y=r, gate=f32(2, 41))):
        with pytest.raises(ValueError):
            ops.block_norm(r, **kw)
    with pytest.raises(TypeError):
        ops.block_norm(r, y=bf(6, 40))
    with pytest.raises(TypeError):
        ops.block_norm(r.double(), w_in=f32(40).double())
    with pytest.raises(ValueError):
        ops.block_norm(r, y=r, out=(r, r))
    with pytest.raises(ValueError, match="required"):
        ops.block_norm(r, y=r, out=(None, None))
    with pytest.raises(ValueError, match=GPU_ONLY):
        ops.block_norm(r, y=r, w_out=f32(40), gate=f32(2, 40), w_in=f32(40))
    for kw in (dict(y=r), dict(y=r, dz=r), dict(y=r, w_in=f32(40), dres_out=r), dict(dres_out=r),
               dict(w_out=f32(40), w_in=f32(40), dz=r), dict(y=r, dres_out=f32(6, 41)), dict(y=r, dres_out=r, out=(r, r)),
               dict(y=r, dres_out=r, out=(r, r, f32(40), None, None)), dict(y=r, dres_out=r, out=(r, None, None, None, None))):
        with pytest.raises(ValueError):
            ops.block_norm_bwd(r, **kw)
    with pytest.raises(ValueError):
        ops.block_norm_bwd(None, w_in=f32(40), dz=r)
    with pytest.raises(ValueError, match=GPU_ONLY):
        ops.block_norm_bwd(r, y=r, w_in=f32(40), dz=r)


def test_exports():
    for name in ("route", "route_bwd", "router", "moe_fwd", "moe_workspace_bytes", "block_norm", "block_norm_bwd",
                 "block_norms", "block_norm_bwd_workspace_bytes"):
        assert name in S.__all__ and callable(getattr(S, name))
