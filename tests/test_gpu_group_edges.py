"""Edges of the operators over rows in order of expert and of the clipping, on the GPU: the tiles that large calls take,
the path of tokens past 32-bit offsets, what a row's result depends on, limits and layouts of clipped gradients.

Bounds as in test_gpu_group.py.
"""
import math

import numpy as np
import pytest
import torch

from oracle import group_oracle as G
from parity_util import BF16_HALF_ULP, U32, check_guards, guarded

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import swiglu_mlp_fwd_amd as S  # noqa: E402
import swiglu_mlp_fwd_amd.group_ops as ops  # noqa: E402
from group_tile_cases import GATED, SINGLE, rows_of  # noqa: E402
from test_gpu_group import DEV, DT, ROUND, block_problem, host, ints, normal, offsets_of, poisoned, within, workspace  # noqa: E402


# ---------------------------------------------------------------- large tiles

@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt,counts,N,K", [c[:4] for c in GATED])
def test_large_tiles_of_the_gate_up_stage(dt, counts, N, K, act):
    """Forward, on rows and with src, and backward, with the large tile (bf16 256 x 128, fp32 128 x 64) over a dozen
    k-steps: which one a case takes is asserted in test_group_edges_host.py."""
    offsets, R, E = offsets_of(counts, 2), rows_of(counts), len(counts)
    x, xc = poisoned(normal((R, K), 1, dt), offsets)
    dh, dhc = poisoned(normal((R, N), 2, dt), offsets)
    wg, wu = normal((E, N, K), 3, dt, K ** -0.5), normal((E, N, K), 4, dt, K ** -0.5)
    o, what = offsets.cpu().numpy(), f"large gate/up {dt} {counts} {N}x{K} {act}"
    h = guarded((R, N), DT[dt])
    S.grouped_fwd(x, wg, wu, offsets, act=act, out=h.t)
    check_guards(what, h)
    within(h.t, *G.gate_up(host(xc), host(wg), host(wu), o, act, ROUND[dt]), what)
    src = torch.arange(R - 1, -1, -1, dtype=torch.int32, device=DEV)
    assert torch.equal(S.grouped_fwd(x.flip(0), wg, wu, offsets, src=src, act=act), h.t)
    out = [guarded(s, DT[dt]) for s in ((R, K), (E, N, K), (E, N, K))]
    S.grouped_bwd(x, wg, wu, dh, offsets, act=act, out=tuple(g.t for g in out))
    check_guards(what, *out)
    want = G.gate_up_bwd(host(xc), host(wg), host(wu), host(dhc), o, act, ROUND[dt])
    for g, (v, b), part in zip(out, want, ("dx", "dwg", "dwu")):
        within(g.t, v, b, f"{what} {part}")


@pytest.mark.parametrize("dt,counts,N,K", [c[:4] for c in SINGLE])
def test_large_tiles_of_the_products(dt, counts, N, K):
    """y = x W^T and dx = dy W, the latter of the product and of both halves of the gate/up stage, with the large tile
    (bf16 256 x 256, fp32 128 x 128) over a dozen k-steps."""
    offsets, R, E = offsets_of(counts, 2), rows_of(counts), len(counts)
    o, what = offsets.cpu().numpy(), f"large product {dt} {counts} {N}x{K}"
    x, xc = poisoned(normal((R, K), 1, dt), offsets)
    w = normal((E, N, K), 3, dt, K ** -0.5)
    y = guarded((R, N), DT[dt])
    S.grouped_mm(x, w, offsets, out=y.t)
    check_guards(what, y)
    within(y.t, *G.mm(host(xc), host(w), o, ROUND[dt]), what)
    # The gradient of rows of N columns, whose reduction is K.
    xb, xbc = poisoned(normal((R, N), 5, dt), offsets)
    wb, wu = normal((E, K, N), 6, dt, N ** -0.5), normal((E, K, N), 7, dt, N ** -0.5)
    out = [guarded((R, N), DT[dt]), guarded((E, K, N), DT[dt])]
    S.grouped_mm_bwd(xb, wb, x, offsets, out=tuple(g.t for g in out))
    check_guards(what, *out)
    for g, (v, b), part in zip(out, G.mm_bwd(host(xbc), host(wb), host(xc), o, ROUND[dt]), ("dx", "dw")):
        within(g.t, v, b, f"{what} {part}")
    dx = guarded((R, N), DT[dt])
    S.grouped_bwd(xb, wb, wu, x, offsets, out=(dx.t, None, None), need_dw=False)
    check_guards(what, dx)
    within(dx.t, *G.gate_up_bwd(host(xbc), host(wb), host(wu), host(xc), o, "silu", ROUND[dt])[0], what + " dx of both halves")


# ------------------------------------------- tokens past 32-bit row offsets

@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_of_large_tokens_gather_them_first(dt, monkeypatch):
    """Tokens of 2^31 bytes and more (the limit is moved down here): the gate/up gradients, in a workspace of either kind,
    and the routed MLP in both directions give the bits that they give below it."""
    (x, wg, wu, wd), logits, dy, k = block_problem(dt)
    w, ids = S.route(logits.detach(), k)
    E, N, K = wg.shape
    offsets, src, _ = S.expert_plan(ids, E)
    R = src.numel()
    dh = normal((R, N), 9, dt)
    leaves = (x, wg, wu, wd, w.requires_grad_(True))

    def passes():
        with torch.no_grad():
            grads = [S.grouped_bwd(x, wg, wu, dh, offsets, src=src, workspace=ws) for ws in
                     (None, workspace(S.grouped_bwd_workspace_bytes(DT[dt], R, N, K, gathered=True)),
                      workspace(S.grouped_bwd_workspace_bytes(DT[dt], R, N, K)))]
            only = [S.grouped_bwd(x, wg, wu, dh, offsets, src=src, need_dw=False)[0],
                    *S.grouped_bwd(x, wg, wu, dh, offsets, src=src, need_dx=False)[1:]]
        y = S.routed_mlp(x, wg, wu, wd, ids, w)
        return [*(t for g in grads for t in g), *only, y.detach(), *torch.autograd.grad((y.float() * dy.float()).sum(), leaves)]
    want = passes()
    gathers = []
    monkeypatch.setattr(ops, "GATHER_BYTES", 64)
    gather = ops.expert_gather
    monkeypatch.setattr(ops, "expert_gather", lambda *a, **kw: gathers.append(1) or gather(*a, **kw))
    got = passes()
    assert len(gathers) == 7                                             # five calls; the routed MLP in each direction
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.isfinite(a).all() and torch.equal(a, b), i


# ------------------------------------------------- what a row's result depends on

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,moved,N,K", [([40, 7, 0, 23, 30], [1, 7, 9, 23, 60], 200, 264), ([3, 2, 4], [1, 2, 6], 1600, 1744),
                                              ([300, 77, 330], [150, 77, 480], 4552, 424), ([1200, 900], [900, 1200], 152, 320)])
def test_a_row_is_the_same_beside_other_rows(dt, counts, moved, N, K):
    """R and E the same: the rows of an expert, and its weights' gradients, have the same bits whatever the other rows hold,
    however they are spread over the experts, and wherever the expert's rows begin."""
    E, R = len(counts), sum(counts)
    keep = [e for e in range(E) if counts[e] == moved[e]] or [None]
    wg, wu = normal((E, N, K), 3, dt, K ** -0.5), normal((E, N, K), 4, dt, K ** -0.5)

    def problem(c, seed):
        o = offsets_of(c)
        x, dy, dh = normal((R, K), seed, dt), normal((R, N), seed + 1, dt), normal((R, N), seed + 2, dt)
        return o, x, dy, dh
    o1, x1, y1, h1 = problem(counts, 10)
    o2, x2, y2, h2 = problem(moved, 20)
    at = []
    for e in range(E):                              # the first rows of each expert in both, all of them where as many
        n = min(counts[e], moved[e])
        a, b = int(o1[e]), int(o2[e])
        for t1, t2 in ((x1, x2), (y1, y2), (h1, h2)):
            t2[b:b + n] = t1[a:a + n]
        at.append((a, b, n))

    def run(x, dy, dh, o):
        y = S.grouped_mm(x, wg, o)
        dx, dw = S.grouped_mm_bwd(x, wg, dy, o)
        return [y, S.grouped_fwd(x, wg, wu, o), dx, S.grouped_bwd(x, wg, wu, dh, o)[0]], [dw, *S.grouped_bwd(x, wg, wu, dh, o)[1:]]
    (rows1, dw1), (rows2, dw2) = run(x1, y1, h1, o1), run(x2, y2, h2, o2)
    for a, b, n in at:
        for i, (t1, t2) in enumerate(zip(rows1, rows2)):
            assert torch.equal(t1[a:a + n], t2[b:b + n]), i
    for e in keep:
        if e is not None:
            for t1, t2 in zip(dw1, dw2):
                assert torch.equal(t1[e], t2[e])


# ------------------------------------------------------------------ clipping

def test_clip_refuses_strided_gradients_that_overlap():
    """As contiguous ones: nothing is written, the shared elements are not counted twice."""
    a = normal((12, 20), 1, "f32")
    keep = a.clone()
    for views in ([a[:, ::2], a[:, ::2]], [a, a[:, ::2]]):
        with pytest.raises(ValueError, match="overlap"):
            S.clip_grads(views, 0.1)
    with pytest.raises(ValueError, match="overlap"):
        S.clip_grads([keep[:, :10], keep[:, 10:]], 0.1, out=[a[:, ::2], a[:, :10]])
    assert torch.equal(a, keep)
    even, odd = a[:, ::2], a[:, 1::2]
    norm, f = G.clip([host(a)], 0.5)
    got = S.clip_grads([even, odd], 0.5)
    assert abs(got.item() - norm) <= 2 * U32 * norm
    within(a, f * host(keep), 3 * U32 * np.abs(host(keep)), "interleaved columns")


@pytest.mark.parametrize("into", [False, True])
def test_clip_limits_without_a_quotient(into):
    """An infinite limit clips nothing, whatever the norm; a norm and eps of zero leave the zeros that there are."""
    def clip(g, limit, **kw):
        out = [torch.full_like(t, 7.0) for t in g] if into else None
        norm = S.clip_grads(g, limit, out=out, **kw)
        return norm.item(), out if into else g
    vals = [torch.tensor([3.0, -math.inf, 0.5], device=DEV), torch.tensor([1.5, -2.0], device=DEV, dtype=torch.bfloat16)]
    norm, got = clip([t.clone() for t in vals], math.inf)
    assert norm == math.inf and all(torch.equal(a, b) for a, b in zip(got, vals))
    zeros = [torch.zeros(9, device=DEV), torch.zeros(5, device=DEV, dtype=torch.bfloat16)]
    for limit in (0.0, 1.0, math.inf):
        norm, got = clip([t.clone() for t in zeros], limit, eps=0.0)
        assert norm == 0.0 and all((t == 0).all() for t in got), limit
    norm, got = clip([torch.tensor([math.nan, 1.0], device=DEV)], math.inf)
    assert math.isnan(norm) and torch.isnan(got[0]).all()                # a step that went wrong stays visible
    norm, got = clip([torch.tensor([3.0, 4.0], device=DEV)], 0.0, eps=0.0)
    assert norm == 5.0 and (got[0] == 0).all()


@pytest.mark.parametrize("into", [False, True])
def test_clip_of_strided_inference_tensors(into):
    """Made in inference mode, clipped outside of it, not contiguous."""
    with torch.inference_mode():
        a, o = torch.full((4, 6), 2.0, device=DEV), torch.zeros((4, 6), device=DEV)
        g, t = a[:, ::2], o[:, ::2]
    plain = torch.full((3,), 2.0, device=DEV)
    S.clip_grads([g, plain], 1.0, eps=0.0, out=[t, plain] if into else None)
    w = 2 / math.sqrt(4 * 15)
    for v in (t if into else g, plain):
        assert (v - w).abs().max().item() <= 2 * U32 * w
    assert (a[:, 1::2] == 2).all() and (o[:, 1::2] == 0).all() and (not into or (a == 2).all())


# ------------------------------------------------------------------ workspace

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", [([3], 13448, 248), ([40] * 5, 1600, 1744), ([3000], 152, 320), ([2000, 40, 2500, 2000], 264, 72),
                                        ([90] * 40, 136, 264)])
def test_gradients_stay_inside_the_workspace_of_their_experts(dt, counts, N, K):
    """Reductions split or not: exactly the bytes asked for, guarded, give the bits that more of them give."""
    offsets, R, E = offsets_of(counts), sum(counts), len(counts)
    x, dy = normal((R, K), 1, dt), normal((R, N), 2, dt)
    wg, wu = normal((E, N, K), 3, dt, K ** -0.5), normal((E, N, K), 4, dt, K ** -0.5)
    src = torch.arange(R, dtype=torch.int32, device=DEV)
    for what, need, call in (
            ("mm", S.grouped_mm_bwd_workspace_bytes(DT[dt], R, N, K, E=E), lambda ws: S.grouped_mm_bwd(x, wg, dy, offsets, workspace=ws)),
            ("gate/up", S.grouped_bwd_workspace_bytes(DT[dt], R, N, K, E=E), lambda ws: S.grouped_bwd(x, wg, wu, dy, offsets, workspace=ws)),
            ("gathered", S.grouped_bwd_workspace_bytes(DT[dt], R, N, K, gathered=True, E=E),
             lambda ws: S.grouped_bwd(x, wg, wu, dy, offsets, src=src, workspace=ws))):
        if need == 0:
            continue
        ws = guarded((need,), torch.uint8)
        got = call(ws.t)
        check_guards(what, ws)
        for a, b in zip(got, call(torch.full((2 * need,), 0xFF, dtype=torch.uint8, device=DEV))):
            assert torch.isfinite(a).all() and torch.equal(a, b), what


# ---------------------------------------------------- past 2^31 elements

def test_rows_past_two_to_the_31_elements():
    """Rows whose elements pass 2^31: gather, product, its gradients, the gate/up stage with src, and combine at their far
    end, by rows that are all zero but for a few."""
    T, K, N, E = (1 << 18) + 5, 8200, 8, 2                              # 2.15e9 elements, 4.3 GB
    g = torch.Generator(device=DEV).manual_seed(1)
    some = torch.tensor([0, 77, T // 2, T - 3, T - 1], device=DEV)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    x[some] = torch.randn((5, K), generator=g, device=DEV).to(torch.bfloat16)
    few = host(x[some])
    split = T - 2
    offsets = ints([0, split, T])
    of = [0, 0, 0, 0, 1]                                                # their experts
    w = normal((E, N, K), 2, "bf16", K ** -0.5)
    want, bound = G.mm(few, host(w), [0, 4, 5], BF16_HALF_ULP)
    y = S.grouped_mm(x, w, offsets)
    within(y[some], want, bound, "far rows: product")
    assert torch.count_nonzero(y).item() == torch.count_nonzero(y[some]).item()
    src = torch.arange(T, dtype=torch.int32, device=DEV)
    assert torch.equal(S.grouped_fwd(x, w, w, offsets, src=src), S.grouped_fwd(x, w, w, offsets))
    dy = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    dy[some] = torch.randn((5, N), generator=g, device=DEV).to(torch.bfloat16)
    dx, dw = S.grouped_mm_bwd(x, w, dy, offsets)
    (wx, bx), (ww, bw) = G.mm_bwd(few, host(w), host(dy[some]), [0, 4, 5], BF16_HALF_ULP)
    within(dx[some], wx, bx, "far rows: dx")
    within(dw, ww, bw, "far rows: dw")
    del dx
    rows = S.expert_gather(x, src.flip(0))
    assert torch.equal(rows[(T - 1 - some).sort().values], x[some.flip(0)])
    pos = src.flip(0).reshape(T, 1)
    wt = torch.full((T, 1), 0.5, device=DEV)
    back = S.expert_combine(rows, pos, wt)
    assert torch.equal(back[some], x[some] * 0.5)                       # a power of two: exact
    del back
    drows, dwt = S.expert_combine_bwd(x, rows, pos, wt)
    assert torch.equal(drows[T - 1 - some], x[some] * 0.5)
    sq = (few * few).sum(1)
    within(dwt[some, 0], sq, 2 * (K + 8) * U32 * sq, "far rows: dweights")
    assert of == [int(r >= split) for r in some.tolist()]


def test_clip_past_two_to_the_31_elements():
    n = (1 << 31) + 12345
    t = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    parts = [t[:7], t[7:n - 3], t[n - 3:]]
    want = 0.5 * math.sqrt(n)
    norm = S.clip_grads(parts, want / 2, eps=0.0)
    assert abs(norm.item() - want) <= 2 ** -23 * want
    assert (t[-(1 << 20):] == 0.25).all() and (t[:1 << 20] == 0.25).all() and t.min().item() == t.max().item() == 0.25
