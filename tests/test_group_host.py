"""Rows in order of expert without a GPU: refusals of the C ABI and of the wrappers, workspace sizes, autograd forms over
stand-ins for the library's calls."""
import ctypes
import math
import os
import shutil
import subprocess
from array import array

import pytest
import torch

import swiglu_mlp_fwd_amd as S
import swiglu_mlp_fwd_amd.group_ops as ops
from test_abi_host import A, EALIGN, EARG, EDTYPE, ENULL, ESHAPE, EUNSUP, EWS, L, MIS, OK  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def a256(n):
    return -(-n // 256) * 256


def test_plan_validation(L):  # noqa: F811
    f, need = L.swiglu_expert_plan, L.swiglu_expert_plan_workspace_bytes
    assert need(1024, 8, 64) == 0 and need(8192, 1, 64) == 0             # one workgroup
    assert need(8193, 1, 64) == a256(9 * 65 * 4) and need(32768, 8, 128) == a256(128 * 129 * 4)
    assert need(-1, 1, 4) == need(1, 0, 4) == need(1, 17, 4) == need(1, 1, 0) == need(1, 1, 1025) == need(1 << 30, 2, 4) == 0

    def call(T=100, k=2, E=8, ids=A, off=A, src=A, pos=A, ws=None, n=0):
        return f(T, k, E, ids, off, src, pos, ws, n, None)
    for bad in (dict(T=-1), dict(k=0), dict(k=17), dict(E=0), dict(E=1025), dict(T=1 << 30), dict(T=1 << 62, k=16)):
        assert call(**bad) == ESHAPE, bad
    for name in ("ids", "off", "src", "pos"):
        assert call(**{name: None}) == ENULL and call(**{name: A + 2}) == EALIGN, name
    assert call(T=0, off=None) == ENULL
    big = dict(T=32768, k=8, E=128)
    n = need(32768, 8, 128)
    assert call(**big) == EWS and call(**big, ws=A, n=n - 1) == EWS and call(**big, ws=A + 64, n=n) == EALIGN


@pytest.mark.parametrize("dt,chunk", [(0, 4), (1, 8)])
def test_rows_validation(L, dt, chunk):  # noqa: F811
    def gather(dt=dt, T=4, k=2, K=64, x=A, src=A, rows=A):
        return L.swiglu_expert_gather(dt, T, k, K, x, src, rows, None)

    def combine(dt=dt, T=4, k=2, K=64, rows=A, pos=A, w=A, y=A):
        return L.swiglu_expert_combine(dt, T, k, K, rows, pos, w, y, None)

    def bwd(dt=dt, T=4, k=2, K=64, dy=A, rows=A, pos=A, w=A, dr=A, dw=A):
        return L.swiglu_expert_combine_bwd(dt, T, k, K, dy, rows, pos, w, dr, dw, None)
    for f in (gather, combine, bwd):
        assert f(dt=2) == EDTYPE
        for bad in (dict(T=-1), dict(k=0), dict(k=17), dict(K=-chunk), dict(K=64 + chunk // 2), dict(T=1 << 31)):
            assert f(**bad) == ESHAPE, bad
        assert f(T=(1 << 23) + 1, k=1) == EUNSUP and f(T=1 << 21, k=16, K=64 * chunk * 2) == EUNSUP
        assert f(T=0, **{n: None for n in ("x", "src", "rows", "pos", "w", "y", "dy", "dr", "dw")
                         if n in f.__code__.co_varnames}) == OK
    for f, names in ((gather, ("x", "rows")), (combine, ("rows", "y")), (bwd, ("dy", "rows", "dr"))):
        for n in names:
            assert f(**{n: None}) == ENULL and f(**{n: MIS}) == EALIGN, n
    for f, n in ((gather, "src"), (combine, "pos"), (bwd, "pos")):
        assert f(**{n: None}) == ENULL and f(**{n: A + 1}) == EALIGN
    assert combine(w=A + 2) == EALIGN and bwd(w=A + 2) == EALIGN and bwd(dw=A + 2) == EALIGN


def grouped_calls(L):  # noqa: F811
    def fwd(act=0, dt=1, R=64, E=4, N=40, K=64, x=A, T=0, k=1, src=None, off=A, wg=A, sg=40 * 64, wu=A, su=40 * 64, h=A):
        return L.swiglu_grouped_fwd(act, dt, R, E, N, K, x, T, k, src, off, wg, sg, wu, su, h, None)

    def bwd(act=0, dt=1, R=64, E=4, N=40, K=64, x=A, T=0, k=1, src=None, off=A, wg=A, sg=40 * 64, wu=A, su=40 * 64,
            dh=A, dx=A, dwg=A, dwu=A, ws=A, n=1 << 40):
        return L.swiglu_grouped_bwd(act, dt, R, E, N, K, x, T, k, src, off, wg, sg, wu, su, dh, dx, dwg, dwu, ws, n, None)

    def mm(dt=1, R=64, E=4, N=40, K=64, x=A, off=A, w=A, sw=40 * 64, y=A):
        return L.swiglu_grouped_mm(dt, R, E, N, K, x, off, w, sw, y, None)

    def mm_bwd(dt=1, R=64, E=4, N=40, K=64, x=A, off=A, w=A, sw=40 * 64, dy=A, dx=A, dw=A,
               ws=A, n=1 << 40):
        return L.swiglu_grouped_mm_bwd(dt, R, E, N, K, x, off, w, sw, dy, dx, dw, ws, n, None)
    return fwd, bwd, mm, mm_bwd


def test_grouped_validation(L):  # noqa: F811
    fwd, bwd, mm, mm_bwd = grouped_calls(L)
    assert fwd(act=2) == EARG and bwd(act=-1) == EARG
    for f in (fwd, bwd, mm, mm_bwd):
        stride = ("sw",) if f in (mm, mm_bwd) else ("sg", "su")
        assert f(dt=2) == EDTYPE
        for bad in (dict(R=-1), dict(R=1 << 31), dict(E=0), dict(E=1025), dict(N=-8), dict(N=44), dict(K=60), dict(K=-8),
                    *({s: v} for s in stride for v in (-8, 40 * 64 - 8, 40 * 64 + 4, 1 << 50))):
            assert f(**bad) == ESHAPE, bad
        assert f(dt=0, N=42) == ESHAPE and f(dt=0, K=62) == ESHAPE
        wide = {s: 1 << 40 for s in stride}
        assert f(N=1 << 21, **wide) == EUNSUP and f(K=1 << 22, **wide) == EUNSUP
        assert f(R=(1 << 31) - 1, N=40000, **wide) == EUNSUP          # too many row tiles
        assert f(E=1024, N=40000, K=40000, **wide) == EUNSUP          # too many weight tiles
        assert f(off=None) == ENULL and f(off=A + 2) == EALIGN
    for f, names in ((fwd, ("x", "wg", "wu", "h")), (bwd, ("x", "wg", "wu", "dh")), (mm, ("x", "w", "y")),
                     (mm_bwd, ("x", "w", "dy"))):
        for n in names:
            assert f(**{n: None}) == ENULL and f(**{n: MIS}) == EALIGN, n
    for n in ("dx", "dwg", "dwu"):
        assert bwd(**{n: MIS}) == EALIGN
    assert bwd(dwg=None) == EARG and bwd(dwu=None) == EARG and bwd(dx=None, dwg=None, dwu=None) == ENULL
    assert mm_bwd(dx=None, dw=None) == ENULL and mm_bwd(dx=MIS) == EALIGN and mm_bwd(dw=MIS) == EALIGN
    # What is not read may be missing.
    assert mm_bwd(dx=None, w=None, dy=None) == ENULL and mm_bwd(dw=None, x=None, dy=None) == ENULL
    # Empty: nothing to enqueue.
    assert fwd(R=0, x=None, off=None, wg=None, wu=None, h=None) == OK and fwd(N=0, sg=0, su=0, h=None) == OK
    assert mm(R=0, x=None, off=None, w=None, y=None) == OK
    assert bwd(K=0, sg=0, su=0, x=None, off=None) == OK and mm_bwd(K=0, sw=0, x=None, off=None) == OK
    assert fwd(E=1, sg=0, su=0, h=None) == ENULL                        # one expert: its stride means nothing


def test_gathered_validation(L):  # noqa: F811
    fwd, bwd, _, _ = grouped_calls(L)
    for f in (fwd, bwd):
        assert f(src=A, T=32, k=2, x=None) == ENULL
        for bad in (dict(T=31, k=2), dict(T=64, k=2), dict(T=-1, k=2), dict(T=32, k=0), dict(T=32, k=17)):
            assert f(src=A, **bad) == ESHAPE, bad
        assert f(src=A + 2, T=32, k=2) == EALIGN
        # Tokens of 2^31 bytes: gather first.
        big = dict(R=1 << 19, T=1 << 19, k=1, K=2048, sg=1 << 30, su=1 << 30)
        assert f(src=A, **big) == EUNSUP


def test_product_gradient_workspace(L):  # noqa: F811
    """The parts' sums of split gradients: many columns or rows to reduce over, few tiles."""
    need = L.swiglu_grouped_mm_bwd_workspace_bytes
    _, _, _, mm_bwd = grouped_calls(L)
    long = dict(R=64, N=4096, K=64, sw=4096 * 64)
    for dt in (0, 1):
        n = need(dt, 64, 4096, 64)
        assert n > 0 and n % 256 == 0 and n % (64 * 64 * 4) == 0
        assert need(dt, 1 << 20, 40, 64) % (40 * 64 * 4) == 0 and need(dt, 1 << 20, 40, 64) > 0
        assert need(dt, 64, 40, 64) == need(dt, 1 << 20, 8192, 8192) == need(dt, 0, 4096, 64) == need(dt, -1, 8, 8) == 0
        assert mm_bwd(dt=dt, ws=None, **long) == EWS and mm_bwd(dt=dt, n=n - 1, **long) == EWS
        assert mm_bwd(dt=dt, ws=A + 128, **long) == EALIGN
        assert S.grouped_mm_bwd_workspace_bytes((torch.float32, torch.bfloat16)[dt], 64, 4096, 64) == n
        assert L.swiglu_grouped_bwd_workspace_bytes(dt, 64, 4096, 64, 0) > 64 * 2 * 4096 * (4, 2)[dt]
    with pytest.raises(TypeError):
        S.grouped_mm_bwd_workspace_bytes(torch.float16, 1, 8, 8)


def test_grouped_workspace(L):  # noqa: F811
    need = L.swiglu_grouped_bwd_workspace_bytes
    _, bwd, _, _ = grouped_calls(L)
    for dt, es in ((0, 4), (1, 2)):
        assert need(dt, 100, 40, 64, 0) == a256(100 * 80 * es)
        assert need(dt, 100, 40, 64, 1) == a256(100 * 80 * es) + a256(100 * 64 * es)
        assert S.grouped_bwd_workspace_bytes((torch.float32, torch.bfloat16)[dt], 100, 40, 64, gathered=True) == need(dt, 100, 40, 64, 1)
    assert need(1, -1, 40, 64, 0) == need(1, 1, 44, 64, 0) == need(2, 1, 40, 64, 0) == 0
    n = need(1, 64, 40, 64, 0)
    assert bwd(ws=None) == EWS and bwd(n=n - 1) == EWS and bwd(ws=A + 128) == EALIGN
    assert bwd(src=A, T=32, k=2, n=n) == EWS                            # the gathered rows want room too
    with pytest.raises(TypeError):
        S.grouped_bwd_workspace_bytes(torch.float16, 1, 8, 8)


def grads(*specs):
    """Host arrays of (dtype, address, size)."""
    d, p, n = array("i", [s[0] for s in specs]), array("Q", [s[1] for s in specs]), array("q", [s[2] for s in specs])
    return d, p, n


def at(a):
    return None if a is None else a.buffer_info()[0]


def test_clip_validation(L):  # noqa: F811
    need = L.swiglu_grad_norm_workspace_bytes
    assert need(0) >= 256 and need(-1) == need((1 << 20) + 1) == 0 and need(641) > need(640)

    def both(specs, outs=None, max_norm=1.0, eps=1e-6, norm=A, ws=A, n=1 << 40, count=None):
        d, p, s = grads(*specs)
        o = None if outs is None else array("Q", outs)
        c = len(specs) if count is None else count
        return L.swiglu_clip_grads(c, at(d), at(p), at(s), at(o), max_norm, eps, norm, ws, n, None)

    def norm_only(specs, norm=A, ws=A, n=1 << 40):
        d, p, s = grads(*specs)
        return L.swiglu_grad_norm(len(specs), at(d), at(p), at(s), norm, ws, n, None)
    one = (0, A, 10)
    for f in (both, norm_only):
        assert f([(2, A, 10)]) == EDTYPE and f([(0, A, -1)]) == ESHAPE and f([(0, A, (1 << 35) + 1)]) == EUNSUP
        assert f([(0, 0, 10)]) == ENULL and f([(0, A + 2, 10)]) == EALIGN and f([(1, A + 1, 10)]) == EALIGN
        assert f([one], norm=None) == ENULL and f([one], norm=A + 2) == EALIGN
        assert f([one], ws=None) == EWS and f([one], n=need(1) - 1) == EWS and f([one], ws=A + 4) == EALIGN
    assert L.swiglu_clip_grads(1, None, None, None, None, 1.0, 1e-6, A, A, 1 << 40, None) == ENULL
    assert both([one], count=-1) == ESHAPE and both([one], count=(1 << 20) + 1) == ESHAPE
    for bad in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf)):
        assert both([one], **bad) == EARG, bad
    # What is written overlaps: the same tensor twice, one inside another, one element shared.
    assert both([one, one]) == EARG and both([(0, A, 10), (1, A + 8, 2)]) == EARG and both([(0, A, 10), (0, A + 36, 10)]) == EARG
    B = A + 0x100000
    assert both([one], outs=[0]) == ENULL and both([one], outs=[B + 2]) == EALIGN
    assert both([one, (0, A + 4096, 10)], outs=[B, B + 36]) == EARG     # outputs overlap
    assert both([one, (0, A + 4096, 10)], outs=[A + 4096, B]) == EARG   # one output is the other's gradient
    assert both([one], outs=[A + 4]) == EARG                            # shifted onto its own


def test_overlap_rules_sanitized(tmp_path):
    """The plan's shares, the overlap rule and the argument checks under the sanitizers; see group_rules_sanitized.cpp."""
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path / "group_rules_sanitized"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "swiglu_mlp_fwd_amd", "csrc"), os.path.join(HERE, "group_rules_sanitized.cpp"),
           "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"build failed:\n{r.stderr}"
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "group rules: ok" in r.stdout, f"{r.stdout}\n{r.stderr}"


# ---------------------------------------------------------------- wrappers

def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_plan_and_rows_wrappers_refuse():
    with pytest.raises(ValueError, match="GPU"):
        S.expert_plan(i32(4, 2), 8)
    for ids, E, err in ((i32(4, 17), 8, ValueError), (i32(4, 0), 8, ValueError), (i32(4, 2), 0, ValueError),
                        (i32(4, 2), 1025, ValueError), (i32(4, 2).long(), 8, TypeError), (torch.tensor(3), 8, ValueError)):
        with pytest.raises(err):
            S.expert_plan(ids, E)
    with pytest.raises(ValueError, match="src"):
        S.expert_plan(i32(4, 2), 8, out=(i32(9), i32(9), i32(4, 2)))
    x = torch.zeros(4, 16)
    for a, src, err in ((x, i32(7), ValueError), (x, i32(4, 2), ValueError), (x, i32(8).long(), TypeError),
                        (x.half(), i32(8), TypeError), (x, i32(4 * 17), ValueError), (x, i32(0), ValueError)):
        with pytest.raises(err):
            S.expert_gather(a, src)
    rows, w = torch.zeros(8, 16), torch.zeros(4, 2)
    for r, pos, ww, err in ((rows[:7], i32(4, 2), w, ValueError), (rows, i32(4, 2).long(), w, TypeError),
                            (rows, i32(4, 2), w[:3], ValueError), (rows, i32(4, 2), w.double(), TypeError),
                            (rows, i32(4, 17), None, ValueError), (rows.half(), i32(4, 2), w, TypeError)):
        with pytest.raises(err):
            S.expert_combine(r, pos, ww)
        with pytest.raises(err):
            S.expert_combine_bwd(torch.zeros(4, 16, dtype=r.dtype), r, pos, ww)
    with pytest.raises(ValueError, match="dy"):
        S.expert_combine_bwd(torch.zeros(8, 16), rows, i32(4, 2), w)
    with pytest.raises(ValueError, match="does not compute"):
        S.expert_combine_bwd(x, rows, i32(4, 2), None, out=(rows.clone(), w))
    with pytest.raises(ValueError, match="pos"):
        S.expert_rows(x, i32(8), i32(8, 1))


def test_grouped_wrappers_refuse():
    x, w, off = torch.zeros(6, 16), torch.zeros(3, 8, 16), i32(4)
    dh = torch.zeros(6, 8)
    bad = [dict(x=x.half()), dict(x=x[:, :8]), dict(x=x[0]), dict(wg=w[0]), dict(wu=w[:2]), dict(off=i32(3)),
           dict(off=i32(4).long()), dict(act="relu"), dict(wg=w.bfloat16()), dict(src=i32(5)), dict(src=i32(12).long())]
    for b in bad:
        kw = {**dict(x=x, wg=w, wu=w, off=off, act="silu", src=None), **b}
        with pytest.raises((ValueError, TypeError)):
            S.grouped_fwd(kw["x"], kw["wg"], kw["wu"], kw["off"], src=kw["src"], act=kw["act"])
        with pytest.raises((ValueError, TypeError)):
            S.grouped_bwd(kw["x"], kw["wg"], kw["wu"], dh, kw["off"], src=kw["src"], act=kw["act"])
    for f in (lambda: S.grouped_fwd(x, w, w, off), lambda: S.grouped_mm(x, w, off),
              lambda: S.grouped_bwd(x, w, w, dh, off), lambda: S.grouped_mm_bwd(x, w, dh, off)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(ValueError, match="dh"):
        S.grouped_bwd(x, w, w, dh[:, :4], off)
    with pytest.raises(ValueError, match="output"):
        S.grouped_bwd(x, w, w, dh, off, need_dx=False, need_dw=False)
    with pytest.raises(ValueError, match="does not compute"):
        S.grouped_bwd(x, w, w, dh, off, need_dx=False, out=(x.clone(), w.clone(), w.clone()))
    with pytest.raises(ValueError, match="contiguous"):
        S.grouped_fwd(x, w, w, off, out=torch.zeros(8, 6).t())
    with pytest.raises(ValueError, match="workspace"):
        S.grouped_bwd(x, w, w, dh, off, workspace=torch.zeros(64, dtype=torch.uint8)[::2])
    with pytest.raises(ValueError, match="dy"):
        S.grouped_mm_bwd(x, w, dh[:5], off)
    with pytest.raises(ValueError, match="output"):
        S.grouped_mm_bwd(x, w, dh, off, need_dx=False, need_dw=False)
    wd, ids, ww = torch.zeros(3, 16, 8), i32(6, 2), torch.zeros(6, 2)
    for args in ((x, w, w, w, ids, ww), (x, w, w, wd, ids[:5], ww), (x, w, w, wd, ids.long(), ww), (x, w, w, wd, ids, ww.double()),
                 (x, w, w, wd, ids, ww[:, :1]), (x[:, :8], w, w, wd, ids, ww), (x, w, w, wd.bfloat16(), ids, ww)):
        with pytest.raises((ValueError, TypeError)):
            S.routed_mlp(*args)
    with pytest.raises(ValueError, match="GPU"):
        S.routed_mlp(x, w, w, wd, ids, ww)


def test_clip_wrapper_refuses():
    a = torch.zeros(4)
    with pytest.raises(ValueError, match="no gradients"):
        S.clip_grads([], 1.0)
    with pytest.raises(TypeError):
        S.clip_grads([a.half()], 1.0)
    with pytest.raises(ValueError, match="out must have"):
        S.clip_grads([a], 1.0, out=[a, a])
    for o in (torch.zeros(5), torch.zeros(4, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match=r"out\[0\]"):
            S.clip_grads([a], 1.0, out=[o])
    with pytest.raises(ValueError, match="share memory"):
        S.clip_grads([torch.zeros(1).expand(4)], 1.0)
    with pytest.raises(ValueError, match="GPU"):
        S.clip_grads([a], 1.0)
    with pytest.raises(ValueError, match="GPU"):
        S.grad_norm(a)


@pytest.mark.parametrize("t,packed,apart", [
    (torch.zeros(3, 4), True, True), (torch.zeros(3, 4).t(), True, True), (torch.zeros(2, 3, 4).permute(2, 0, 1), True, True),
    (torch.zeros(3, 8)[:, ::2], False, True), (torch.zeros(3, 8)[:, :4], False, True), (torch.zeros(4).expand(3, 4), False, False),
    (torch.zeros(9).as_strided((3, 3), (2, 1)), False, False), (torch.zeros(1, 5)[:, :1], True, True), (torch.zeros(()), True, True)])
def test_how_elements_lie(t, packed, apart):
    assert ops._packed(t) == packed and ops._apart(t) == apart


# -------------------------------------------------- autograd over stand-ins

@torch.no_grad()
def plain_mm(x, w, offsets, out=None):
    return torch.cat([x[a:b] @ w[e].t() for e, (a, b) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:]))])


@torch.no_grad()
def plain_mm_bwd(x, w, dy, offsets, out=None, need_dx=True, need_dw=True):
    at_ = list(zip(offsets.tolist(), offsets.tolist()[1:]))
    dx = torch.cat([dy[a:b] @ w[e] for e, (a, b) in enumerate(at_)]) if need_dx else None
    dw = torch.stack([dy[a:b].t() @ x[a:b] for a, b in at_]) if need_dw else None
    return dx, dw


def test_grouped_linear_over_a_stand_in(monkeypatch):
    monkeypatch.setattr(ops, "grouped_mm", plain_mm)
    monkeypatch.setattr(ops, "grouped_mm_bwd", plain_mm_bwd)
    x, w = torch.randn(7, 5, requires_grad=True), torch.randn(3, 4, 5, requires_grad=True)
    off = torch.tensor([0, 2, 2, 7], dtype=torch.int32)
    y = ops.grouped_linear(x, w, off)
    dy = torch.randn_like(y)
    got = torch.autograd.grad((y * dy).sum(), (x, w))
    for a, b in zip(got, plain_mm_bwd(x, w, dy, off)):
        assert torch.equal(a, b)
    y = ops.grouped_linear(x.detach(), w, off)               # x needs none
    assert torch.equal(torch.autograd.grad((y * dy).sum(), w)[0], got[1])
    (d,) = torch.autograd.grad(ops.grouped_linear(x, w, off).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        d.square().sum().backward()


def test_routed_mlp_forms_the_gradients_it_needs(monkeypatch):
    """Which of the pieces are called for which inputs, and where their results go."""
    calls = []
    T, k, E, N, K = 3, 2, 2, 4, 5
    R = T * k

    def note(name, value):
        def f(*a, **kw):
            calls.append((name, kw.get("need_dx"), kw.get("need_dw")))
            return value(kw)
        return f
    z = torch.zeros
    monkeypatch.setattr(ops, "_on_gpu", lambda t: None)
    monkeypatch.setattr(ops, "expert_plan", note("plan", lambda kw: (i32(E + 1), i32(R), i32(T, k))))
    monkeypatch.setattr(ops, "grouped_fwd", note("fwd", lambda kw: z(R, N)))
    monkeypatch.setattr(ops, "grouped_mm", note("mm", lambda kw: z(R, K)))
    monkeypatch.setattr(ops, "expert_combine", note("combine", lambda kw: torch.full((T, K), 7.0)))
    monkeypatch.setattr(ops, "expert_combine_bwd", note("combine_bwd", lambda kw: (z(R, K), torch.full((T, k), 2.0))))
    monkeypatch.setattr(ops, "grouped_mm_bwd", note("mm_bwd", lambda kw: (
        z(R, N) if kw["need_dx"] else None, torch.full((E, K, N), 3.0) if kw["need_dw"] else None)))
    monkeypatch.setattr(ops, "grouped_bwd", note("bwd", lambda kw: (
        z(R, K) if kw["need_dx"] else None, *(torch.full((E, N, K), v) if kw["need_dw"] else None for v in (4.0, 5.0)))))
    shapes = dict(x=(T, K), wg=(E, N, K), wu=(E, N, K), wd=(E, K, N), w=(T, k))
    value = dict(x=7.0, wg=4.0, wu=5.0, wd=3.0, w=2.0)
    for keep, want in ((("x", "wg", "wu", "wd", "w"), [("combine_bwd", None, None), ("mm_bwd", True, True), ("bwd", True, True), ("combine", None, None)]),
                       (("x",), [("combine_bwd", None, None), ("mm_bwd", True, False), ("bwd", True, False), ("combine", None, None)]),
                       (("wu",), [("combine_bwd", None, None), ("mm_bwd", True, False), ("bwd", False, True)]),
                       (("wd", "w"), [("combine_bwd", None, None), ("mm_bwd", False, True)]),
                       (("w",), [("combine_bwd", None, None)])):
        t = {n: z(s).requires_grad_(n in keep) for n, s in shapes.items()}
        calls.clear()
        y = ops.routed_mlp(t["x"], t["wg"], t["wu"], t["wd"], i32(T, k), t["w"])
        assert [c[0] for c in calls] == ["plan", "fwd", "mm", "combine"]
        calls.clear()
        y.sum().backward()
        assert calls == want, keep
        for n in shapes:
            assert (t[n].grad is None) == (n not in keep) and (t[n].grad is None or (t[n].grad == value[n]).all())
