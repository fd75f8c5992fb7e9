"""Edges of the operators over rows in order of expert and of the clipping, without a GPU."""
import os
import random
import shutil
import subprocess

import pytest
import torch

import swiglu_mlp_fwd_amd as S
import swiglu_mlp_fwd_amd.group_ops as ops
from group_tile_cases import queries
from test_abi_host import A, EALIGN, EARG, EWS, L  # noqa: F401
from test_group_host import HERE, ROOT, at, grads, grouped_calls


# ------------------------------------------------- how a tensor's elements lie

@pytest.mark.parametrize("t,apart", [
    (torch.zeros(5, 7, 8)[:, ::2, :3], True), (torch.zeros(5, 7, 8)[:, ::2, ::3], True), (torch.zeros(4, 9)[:, ::4], True),
    (torch.zeros(20).as_strided((3, 4), (4, 1)), True), (torch.zeros(20).as_strided((3, 4), (3, 1)), False),
    (torch.zeros(20).as_strided((4, 2, 2), (3, 2, 1)), False)])
def test_slices_that_end_inside_a_stride_are_apart(t, apart):
    """The steps behind a dimension's last element are nobody's: strides (56, 16, 1) of 5 x 4 x 3 elements share none."""
    assert ops._apart(t) == apart
    with pytest.raises(ValueError, match="GPU" if apart else "share memory"):
        S.clip_grads([t], 1.0)


# -------------------------------------- strided gradients that share memory

def columns():
    return torch.zeros(12, 20)


def shares(f, *views):
    with pytest.raises(ValueError, match="overlap"):
        f(*views)


def test_strided_gradients_that_overlap_are_refused():
    a = columns()
    for views in ([a[:, ::2], a[:, ::2]], [a, a[:, ::2]], [a[:, ::2], a[:, 4:7]], [a[::3, 5:9], a[:, 8:]], [a[:, :3], a[2:4, 2:5]],
                  [a[:, ::2], torch.zeros(5), a[3, 4:5]], [a[:, 1:3], a.view(torch.bfloat16)[:, 5:7]]):
        shares(S.clip_grads, views, 1.0)


def test_strided_outputs_that_overlap_are_refused():
    a, b, c = columns(), columns(), torch.zeros(12, 10)
    shares(lambda *v: S.clip_grads([c, c.clone()], 1.0, out=list(v)), a[:, ::2], a[:, :10])      # another output
    shares(lambda *v: S.clip_grads([a[:, 10:], b[:, 10:]], 1.0, out=list(v)), b[:, 10:], c)      # another's gradient
    shares(lambda *v: S.clip_grads([a[:, ::2]], 1.0, out=list(v)), a[:, 1:11])                   # its own, shifted
    square = torch.zeros(6, 6)
    shares(lambda *v: S.clip_grads([square[:4, :4]], 1.0, out=list(v)), square[:4, :4].t())      # its own, otherwise laid out


def test_strided_gradients_that_interleave_are_taken():
    """Spans that cross without a shared element: the call goes as far as the check for a GPU."""
    a = columns()
    deep = torch.zeros(5, 7, 8)
    for views in ([a[:, ::2], a[:, 1::2]], list(a.split([4, 7, 9], 1)), list(deep.unbind(1)), list(deep.unbind(2)),
                  [a[::2], a[1::2]], [a[:, ::2], a[:, 1::4], a[:, 3::4]], [deep[:, ::2, :3], deep[:, 1::2], deep[:, ::2, 3:]],
                  [a[:, 1:3], a.view(torch.bfloat16)[:, 6:8]]):
        with pytest.raises(ValueError, match="GPU"):
            S.clip_grads(views, 1.0)
    for g, out in ((a[:, ::2], a[:, ::2]), (a[:, ::2], a[:, 1::2]), (a.t(), a.t())):
        with pytest.raises(ValueError, match="GPU"):
            S.clip_grads([g], 1.0, out=[out])


def places(t):
    """Byte addresses of t's elements."""
    at = {t.data_ptr()}
    for n, s in zip(t.shape, t.stride()):
        at = {p + i * s * t.element_size() for p in at for i in range(n)} if n else set()
    return {p + b for p in at for b in range(t.element_size())}


def test_overlap_of_random_views_against_all_their_bytes():
    r = random.Random(3)
    flat = torch.zeros(400)
    found = 0
    for _ in range(12000):
        views = []
        for _ in range(r.randint(2, 4)):
            base = flat.view(torch.bfloat16) if r.random() < 0.4 else flat
            while True:
                shape = [r.randint(1, 5) for _ in range(r.randint(0, 3))]
                stride = [r.choice([1, 2, 3, 4, 6, 8, 12, 20, 24, 40]) for _ in shape]
                span = sum((n - 1) * s for n, s in zip(shape, stride)) + 1
                if span <= 100:
                    break
            views.append(base.as_strided(shape, stride, r.randint(0, 260 - span)))
        if not all(map(ops._apart, views)):
            continue
        seen = [places(v) for v in views]
        want = any(seen[i] & seen[j] for i in range(len(views)) for j in range(i))
        found += want
        assert (ops._overlap(views) is not None) == want, [(v.data_ptr(), v.shape, v.stride(), v.dtype) for v in views]
    assert found > 500


def test_norm_and_workspace_inside_a_gradient_are_refused(L):  # noqa: F811
    """They are written too.  (Refused on the host: no address is read.)"""
    far, ws = A + (1 << 24), A + (1 << 25)
    n = L.swiglu_grad_norm_workspace_bytes(2)

    def clip(norm=far, ws=ws, outs=None):
        d, p, s = grads((0, A, 1000), (1, A + 8192, 1000))
        o = None if outs is None else grads(*((0, a, 0) for a in outs))[1]
        return L.swiglu_clip_grads(2, at(d), at(p), at(s), at(o), 1.0, 1e-6, norm, ws, n, None)
    for norm in (A, A + 3996, A + 8192, A + 8192 + 1996):
        assert clip(norm=norm) == EARG, norm - A
        assert clip(norm=norm, outs=(A + 65536, A + 131072)) == EARG, norm - A
    for w in (A, A + 8192 + 1792, A - n + 256):
        assert clip(ws=w) == EARG, w - A
    assert clip(norm=ws + n - 4) == EARG and clip(norm=A + 65536, outs=(A + 65536, A + 131072)) == EARG


# ------------------------------------------------------------------ workspace

def test_gradients_ask_for_the_workspace_that_they_use(L):  # noqa: F811
    """For E experts: parts' sums only where a gradient of so many is split; never more than for any number."""
    fine = dict(R=32768, N=1024, K=2048)
    D, rows = 32768 * 2 * 1024 * 2, 32768 * 2048 * 2
    any_e, of = S.grouped_bwd_workspace_bytes, S.grouped_mm_bwd_workspace_bytes
    assert any_e(torch.bfloat16, **fine, gathered=True, E=64) == D + rows
    assert any_e(torch.bfloat16, **fine, gathered=True) == D + rows + (64 << 20)
    assert any_e(torch.bfloat16, **fine, E=64) == D and of(torch.bfloat16, **fine, E=64) == 0 < of(torch.bfloat16, **fine)
    fwd, bwd, mm, mm_bwd = grouped_calls(L)
    sizes = dict(E=64, **fine, sg=1024 * 2048, su=1024 * 2048)
    assert bwd(**sizes, n=D - 1) == EWS and bwd(**sizes, src=A, T=4096, k=8, n=D + rows - 1) == EWS
    long = dict(E=3, R=64, N=4096, K=64, sw=4096 * 64)
    for dt in (0, 1):
        n = L.swiglu_grouped_mm_bwd_workspace_bytes_of(dt, 64, 3, 4096, 64)
        assert 0 < n <= L.swiglu_grouped_mm_bwd_workspace_bytes(dt, 64, 4096, 64)
        assert mm_bwd(dt=dt, n=n - 1, **long) == EWS and mm_bwd(dt=dt, n=n, ws=A + 128, **long) == EALIGN
    for bad in ((2, 64, 3, 4096, 64), (1, -1, 3, 8, 8), (1, 64, 0, 8, 8), (1, 64, 1025, 8, 8), (1, 64, 3, 4, 8)):
        assert L.swiglu_grouped_mm_bwd_workspace_bytes_of(*bad) == L.swiglu_grouped_bwd_workspace_bytes_of(*bad, 0) == 0
    r = random.Random(1)
    for _ in range(3000):
        dt, E = r.randint(0, 1), r.choice([1, 2, 3, 8, 39, 64, 1024])
        R, N, K = int(2 ** r.uniform(0, 20)), 8 * int(2 ** r.uniform(0, 11)), 8 * int(2 ** r.uniform(0, 11))
        assert L.swiglu_grouped_bwd_workspace_bytes_of(dt, R, E, N, K, 0) <= L.swiglu_grouped_bwd_workspace_bytes(dt, R, N, K, 0) \
            or L.swiglu_grouped_bwd_workspace_bytes(dt, R, N, K, 0) == 0


# ---------------------------------------------------------------------- tiles

def test_large_cases_take_the_tiles_they_name(tmp_path):
    """The sizes that the GPU tests of the large tiles use, by the rules the launches go by; and every launch of allowed
    sizes holds its threads (group_tiles_sanitized.cpp)."""
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path / "group_tiles_sanitized"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-include", "cmath", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "swiglu_mlp_fwd_amd", "csrc"), os.path.join(HERE, "group_tiles_sanitized.cpp"),
           "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"build failed:\n{r.stderr}"
    asked = list(queries())
    lines = "".join(f"{form} {('f32', 'bf16').index(dt)} {R} {E} {n} {red} {halves}\n"
                    for form, dt, R, E, n, red, halves, _, _ in asked)
    r = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "group tiles: ok" in r.stdout, f"{r.stdout}\n{r.stderr}"
    for q, line in zip(asked, r.stdout.splitlines()):
        bm, bn, parts, apart = map(int, line.split())
        assert ((bm, bn), parts, bool(apart)) == (q[7], 1, q[8]), q
