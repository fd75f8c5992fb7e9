"""Rows in order of expert on the GPU against the fp64 oracle: plan, gather, combine, grouped products and their
gradients, the routed MLP as a whole, and the clipping of gradients.

Bounds: oracle/group_oracle.py for the products (propagated fp32 accumulation, the outputs' and [dg | du]'s rounding,
a factor 2 of headroom).  combine: k + 1 fp32 roundings of its absolute terms, and the output's.  dweights: a dot of K
products, each passing at most K additions: (K + 8) u of the absolute terms.  The norm: fp64 sums of exact squares,
rounded once to fp32.
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

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": BF16_HALF_ULP, "f32": U32}


def normal(shape, seed, dt, std=1.0):
    a = np.asarray(np.random.default_rng(seed).normal(size=shape) * std)
    return torch.from_numpy(a).to(torch.float32).to(DT[dt]).to(DEV)


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    got = host(got)
    assert got.shape == want.shape, what
    err = np.abs(got - want)
    assert np.isfinite(got).all(), f"{what}: not finite"
    b = np.broadcast_to(bound, want.shape) + 1e-30
    worst = float((err / b).max()) if err.size else 0.0
    print(f"{what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def offsets_of(counts, first=0):
    return ints(first + np.concatenate([[0], np.cumsum(counts)]))


# ------------------------------------------------------------------ plan

def check_plan(ids, E, what):
    T, k = ids.shape
    out = [guarded((E + 1,), torch.int32), guarded((T * k,), torch.int32), guarded((T, k), torch.int32)]
    S.expert_plan(ids, E, out=tuple(g.t for g in out))
    check_guards(what, *out)
    for g, want, name in zip(out, G.plan(ids.cpu().numpy(), E), ("offsets", "src", "pos")):
        assert np.array_equal(g.t.cpu().numpy(), want), f"{what}: {name}"


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 16, 16), (3, 2, 5), (64, 8, 64), (511, 2, 63), (512, 16, 1024),
                                   (513, 16, 64), (4096, 2, 65), (8193, 1, 3), (20001, 1, 1024), (5003, 7, 127),
                                   (9001, 16, 200)])
def test_plan(T, k, E):
    g = np.random.default_rng(T * 31 + E)
    ids = g.integers(0, E, size=(T, k))
    check_plan(ints(ids).reshape(T, k), E, f"plan {T}x{k} of {E}")
    gone = g.uniform(size=ids.shape)
    ids[gone < 0.2] = -1
    ids[gone > 0.95] = E + 3
    ids[(gone > 0.94) & (gone < 0.95)] = -(1 << 31)
    check_plan(ints(ids).reshape(T, k), E, f"plan {T}x{k} of {E}, dropped")
    check_plan(ints(np.full((T, k), -1)).reshape(T, k), E, f"plan {T}x{k} of {E}, all dropped")
    check_plan(ints(np.full((T, k), E - 1)).reshape(T, k), E, f"plan {T}x{k} of {E}, all on one")


def test_plan_of_slices_and_leading_dimensions():
    ids = torch.randint(0, 9, (6, 10, 4), device=DEV, dtype=torch.int32)
    want = S.expert_plan(ids[:, ::2, 1:3].contiguous().reshape(-1, 2), 9)
    got = S.expert_plan(ids[:, ::2, 1:3], 9)
    assert got[2].shape == (6, 5, 2)
    for a, b in zip(got, want):
        assert torch.equal(a.reshape(-1), b.reshape(-1))


# --------------------------------------------------------- rows and tokens

SHAPES = [(1, 1, 3, 8), (3, 2, 5, 72), (7, 16, 20, 264), (65, 3, 4, 512), (130, 8, 64, 520), (33, 5, 7, 2056),
          (5, 9, 11, 8200)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,K", SHAPES)
def test_gather_and_combine(T, k, E, K, dt):
    g = np.random.default_rng(K)
    ids = g.integers(0, E, size=(T, k))
    ids[g.uniform(size=ids.shape) < 0.15] = -1
    _, src, pos = G.plan(ids, E)
    R = T * k
    x = normal((T, K), 1, dt)
    out = guarded((R, K), DT[dt])
    S.expert_gather(x, ints(src), out=out.t)
    check_guards("gather", out)
    assert np.array_equal(host(out.t), G.gather(host(x), src, k))

    rows, w = normal((R, K), 2, dt), torch.rand((T, k), device=DEV) + 0.1
    rows[torch.as_tensor(src < 0, device=DEV)] = math.nan              # rows of dropped pairs are not read
    for weights in (w, None):
        what = f"combine {T}x{k}x{K} {dt}{'' if weights is None else ' weighted'}"
        wh = None if weights is None else host(weights)
        clean = np.nan_to_num(host(rows))
        y = guarded((T, K), DT[dt])
        S.expert_combine(rows, ints(pos), weights, out=y.t)
        check_guards(what, y)
        want, a = G.combine(clean, pos, wh)
        within(y.t, want, 2 * ((k + 1) * U32 * a + ROUND[dt] * np.abs(want)), what)
        dy = normal((T, K), 3, dt)
        dr, dw = guarded((R, K), DT[dt]), guarded((T, k), torch.float32)
        S.expert_combine_bwd(dy, rows, ints(pos), weights, out=(dr.t, dw.t if weights is not None else None))
        check_guards(what, dr, dw)
        want_r, want_w, aw = G.combine_bwd(host(dy), clean, pos, wh)
        within(dr.t, want_r, 2 * (U32 + ROUND[dt]) * np.abs(want_r), what + " drows")
        if weights is not None:
            within(dw.t, want_w, 2 * (K + 8) * U32 * aw, what + " dweights")


# --------------------------------------------------------- grouped products

# (rows of each expert, rows in front of them, rows behind)
GROUPS = {
    "one": ([1], 0, 0),
    "few": ([3, 0, 1, 5], 0, 0),
    "ragged": ([0, 17, 1, 0, 70, 130, 0], 0, 9),
    "tiles": ([255, 256, 257, 64, 65], 0, 0),
    "slice": ([40, 0, 100], 33, 60),
    "empty": ([0, 0], 0, 5),
    "large": ([600, 2, 301], 0, 1),
}


def sizes(name):
    counts, head, tail = GROUPS[name]
    return counts, offsets_of(counts, head), head + sum(counts) + tail


def poisoned(t, offsets):
    """t with NaN in the rows of no expert, and without them."""
    o = offsets.tolist()
    t = t.clone()
    clean = t.clone()
    t[:o[0]], t[o[-1]:] = math.nan, math.nan
    clean[:o[0]], clean[o[-1]:] = 0, 0
    return t, clean


def workspace(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)       # NaN, whatever is read of it unwritten


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(8, 8), (200, 264), (264, 72), (520, 328)])
@pytest.mark.parametrize("name", GROUPS)
def test_grouped_mm(name, N, K, dt):
    counts, offsets, R = sizes(name)
    E = len(counts)
    x, xc = poisoned(normal((R, K), 1, dt), offsets)
    dy, dyc = poisoned(normal((R, N), 2, dt), offsets)
    w = normal((E, N, K), 3, dt, K ** -0.5)
    what = f"grouped_mm {name} {N}x{K} {dt}"
    y = guarded((R, N), DT[dt])
    S.grouped_mm(x, w, offsets, out=y.t)
    check_guards(what, y)
    o = offsets.cpu().numpy()
    within(y.t, *G.mm(host(xc), host(w), o, ROUND[dt]), what)
    dx, dw = guarded((R, K), DT[dt]), guarded((E, N, K), DT[dt])
    S.grouped_mm_bwd(x, w, dy, offsets, out=(dx.t, dw.t))
    check_guards(what, dx, dw)
    want_x, want_w = G.mm_bwd(host(xc), host(w), host(dyc), o, ROUND[dt])
    within(dx.t, *want_x, what + " dx")
    within(dw.t, *want_w, what + " dw")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(8, 8), (200, 264), (264, 72), (520, 328)])
@pytest.mark.parametrize("name", GROUPS)
def test_grouped_gate_up(name, N, K, dt, act):
    counts, offsets, R = sizes(name)
    E = len(counts)
    x, xc = poisoned(normal((R, K), 1, dt), offsets)
    dh, dhc = poisoned(normal((R, N), 2, dt), offsets)
    wg, wu = normal((E, N, K), 3, dt, K ** -0.5), normal((E, N, K), 4, dt, K ** -0.5)
    what = f"grouped {name} {N}x{K} {dt} {act}"
    h = guarded((R, N), DT[dt])
    S.grouped_fwd(x, wg, wu, offsets, act=act, out=h.t)
    check_guards(what, h)
    o = offsets.cpu().numpy()
    within(h.t, *G.gate_up(host(xc), host(wg), host(wu), o, act, ROUND[dt]), what)
    out = [guarded((R, K), DT[dt]), guarded((E, N, K), DT[dt]), guarded((E, N, K), DT[dt])]
    S.grouped_bwd(x, wg, wu, dh, offsets, act=act, out=tuple(g.t for g in out),
                  workspace=workspace(S.grouped_bwd_workspace_bytes(DT[dt], R, N, K)))
    check_guards(what, *out)
    want = G.gate_up_bwd(host(xc), host(wg), host(wu), host(dhc), o, act, ROUND[dt])
    for g, (v, b), part in zip(out, want, ("dx", "dwg", "dwu")):
        within(g.t, v, b, f"{what} {part}")


def many_tiles(dt):
    """Rows, and a width, whose tiles are more than the CUs, where the launches take their large tiles: many small ragged
    experts (bf16), few large ones (fp32)."""
    g = np.random.default_rng(3)
    counts = list(g.integers(0, 90, size=40)) if dt == "bf16" else [700, 0, 301, 900]
    counts[1] = 300 if dt == "bf16" else 0
    return counts, offsets_of(counts, 2), 2 + int(sum(counts)) + 3


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("wide_first", [True, False])
def test_many_tiles(dt, wide_first):
    """N wide: the products of rows take many tiles; K wide: their gradients."""
    counts, offsets, R = many_tiles(dt)
    E, wide, narrow = len(counts), 2312, 136
    N, K = (wide, narrow) if wide_first else (narrow, wide)
    x, xc = poisoned(normal((R, K), 1, dt), offsets)
    dy, dyc = poisoned(normal((R, N), 2, dt), offsets)
    wg, wu = normal((E, N, K), 3, dt, K ** -0.5), normal((E, N, K), 4, dt, K ** -0.5)
    o = offsets.cpu().numpy()
    hx, hdy, hg, hu = host(xc), host(dyc), host(wg), host(wu)
    out = [guarded(s, DT[dt]) for s in ((R, N), (R, K), (E, N, K), (R, N), (R, K), (E, N, K), (E, N, K))]
    S.grouped_mm(x, wg, offsets, out=out[0].t)
    S.grouped_mm_bwd(x, wg, dy, offsets, out=(out[1].t, out[2].t))
    S.grouped_fwd(x, wg, wu, offsets, out=out[3].t)
    S.grouped_bwd(x, wg, wu, dy, offsets, out=tuple(g.t for g in out[4:]),
                  workspace=workspace(S.grouped_bwd_workspace_bytes(DT[dt], R, N, K)))
    check_guards("many tiles", *out)
    want = [G.mm(hx, hg, o, ROUND[dt]), *G.mm_bwd(hx, hg, hdy, o, ROUND[dt]), G.gate_up(hx, hg, hu, o, "silu", ROUND[dt]),
            *G.gate_up_bwd(hx, hg, hu, hdy, o, "silu", ROUND[dt])]
    for g, (v, b), name in zip(out, want, ("y", "dx", "dw", "h", "dx gate/up", "dwg", "dwu")):
        within(g.t, v, b, f"many tiles {dt} {N}x{K} {name}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_hundreds_of_experts(dt):
    """More groups than a wave has lanes: the scan over them takes several turns."""
    g = np.random.default_rng(9)
    counts = list(g.integers(0, 4, size=1024))
    counts[700] = 90
    offsets, R, N, K = offsets_of(counts, 1), 1 + int(sum(counts)) + 2, 24, 40
    x, xc = poisoned(normal((R, K), 1, dt), offsets)
    dy, dyc = poisoned(normal((R, N), 2, dt), offsets)
    w, o = normal((1024, N, K), 3, dt, K ** -0.5), offsets.cpu().numpy()
    within(S.grouped_mm(x, w, offsets), *G.mm(host(xc), host(w), o, ROUND[dt]), f"1024 experts {dt} y")
    got = S.grouped_mm_bwd(x, w, dy, offsets)
    for t, want, name in zip(got, G.mm_bwd(host(xc), host(w), host(dyc), o, ROUND[dt]), ("dx", "dw")):
        within(t, *want, f"1024 experts {dt} {name}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", [([3], 13448, 248), ([2, 1], 4104, 8), ([0, 70, 0, 3], 2056, 264),
                                        ([40] * 5, 1600, 1744), ([1] * 39, 4928, 72), ([130], 1024, 512)])
def test_split_reduction(dt, counts, N, K):
    """dx of few rows: the reduction over N in parts, with rows of no expert in front and behind."""
    offsets, R, E = offsets_of(counts, 2), 2 + sum(counts) + 3, len(counts)
    x, xc = poisoned(normal((R, K), 1, dt), offsets)
    dy, dyc = poisoned(normal((R, N), 2, dt), offsets)
    wg, wu, o = normal((E, N, K), 3, dt, K ** -0.5), normal((E, N, K), 4, dt, K ** -0.5), offsets.cpu().numpy()
    ws = workspace(S.grouped_mm_bwd_workspace_bytes(DT[dt], R, N, K))
    dx = guarded((R, K), DT[dt])
    S.grouped_mm_bwd(x, wg, dy, offsets, out=(dx.t, None), need_dw=False, workspace=ws)
    check_guards("split product", dx)
    within(dx.t, *G.mm_bwd(host(xc), host(wg), host(dyc), o, ROUND[dt])[0], f"product dx {dt} {counts} {N} {K}")
    assert torch.equal(dx.t, S.grouped_mm_bwd(x, wg, dy, offsets, need_dw=False)[0])
    ws = workspace(S.grouped_bwd_workspace_bytes(DT[dt], R, N, K))
    dx = guarded((R, K), DT[dt])
    S.grouped_bwd(x, wg, wu, dy, offsets, out=(dx.t, None, None), need_dw=False, workspace=ws)
    check_guards("split gate/up", dx)
    within(dx.t, *G.gate_up_bwd(host(xc), host(wg), host(wu), host(dyc), o, "silu", ROUND[dt])[0],
           f"gate/up dx {dt} {counts} {N} {K}")
    assert torch.equal(dx.t, S.grouped_bwd(x, wg, wu, dy, offsets, need_dw=False)[0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", [([3000], 152, 320), ([1, 6000, 0], 8, 264), ([2000, 40, 2500, 2000], 264, 72)])
def test_split_rows(dt, counts, N, K):
    """dW of small weights: each expert's rows in parts, some of them without any."""
    offsets, R, E = offsets_of(counts, 2), 2 + sum(counts) + 3, len(counts)
    x, xc = poisoned(normal((R, K), 1, dt), offsets)
    dy, dyc = poisoned(normal((R, N), 2, dt), offsets)
    wg, wu, o = normal((E, N, K), 3, dt, K ** -0.5), normal((E, N, K), 4, dt, K ** -0.5), offsets.cpu().numpy()
    dw = [guarded((E, N, K), DT[dt]) for _ in range(3)]
    S.grouped_mm_bwd(x, wg, dy, offsets, out=(None, dw[0].t), need_dx=False,
                     workspace=workspace(S.grouped_mm_bwd_workspace_bytes(DT[dt], R, N, K)))
    S.grouped_bwd(x, wg, wu, dy, offsets, out=(None, dw[1].t, dw[2].t), need_dx=False,
                  workspace=workspace(S.grouped_bwd_workspace_bytes(DT[dt], R, N, K)))
    check_guards("split rows", *dw)
    want = [G.mm_bwd(host(xc), host(wg), host(dyc), o, ROUND[dt])[1],
            *G.gate_up_bwd(host(xc), host(wg), host(wu), host(dyc), o, "silu", ROUND[dt])[1:]]
    for g, w, name in zip(dw, want, ("dw", "dwg", "dwu")):
        within(g.t, *w, f"{name} {dt} {counts} {N} {K}")
    assert torch.equal(dw[0].t, S.grouped_mm_bwd(x, wg, dy, offsets)[1])
    assert all(torch.equal(a.t, b) for a, b in zip(dw[1:], S.grouped_bwd(x, wg, wu, dy, offsets)[1:]))


def test_more_small_tiles_than_a_launch_has():
    """Many experts of very many columns: small row and column tiles would be past 2^32 threads."""
    E, N, K, R = 252, (1 << 21) - 32, 8, 255        # (the most rows that 252 experts of as many columns may have)
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
    w[3, -1] = w[251, 0] = 1.0
    x = torch.ones((R, K), dtype=torch.bfloat16, device=DEV)
    h = S.grouped_fwd(x, w, w, offsets_of([1] * E))
    at = torch.nonzero(h.view(torch.int16))
    assert at.tolist() == [[3, N - 1], [251, 0]]
    assert abs(h[3, -1].item() - 64 / (1 + math.exp(-8))) <= 64 * 2 ** -8


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_offsets_that_decrease_stay_inside(dt):
    """Offsets no plan gives (decreasing, negative, past the rows): nothing outside the outputs is touched, and the
    following call is as ever."""
    R, E, N, K = 300, 4, 72, 136
    x, w, dy = normal((R, K), 1, dt), normal((E, N, K), 2, dt), normal((R, N), 3, dt)
    for bad in ([0, 200, 100, 400, 300], [300, 0, 300, 0, 300], [-5, -1, 0, 1 << 30, 10], [(1 << 31) - 1] * 5):
        o = ints(bad)
        out = [guarded(s, DT[dt]) for s in ((R, N), (R, K), (E, N, K), (R, N), (R, K), (E, N, K), (E, N, K))]
        S.grouped_mm(x, w, o, out=out[0].t)
        S.grouped_mm_bwd(x, w, dy, o, out=(out[1].t, out[2].t))
        S.grouped_fwd(x, w, w, o, out=out[3].t)
        S.grouped_bwd(x, w, w, dy, o, out=tuple(g.t for g in out[4:]))
        check_guards(f"offsets {bad}", *out)
    good = offsets_of([100, 0, 150, 50])
    within(S.grouped_mm(x, w, good), *G.mm(host(x), host(w), good.cpu().numpy(), ROUND[dt]), "after bad offsets")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_indices_no_plan_gives(dt):
    """src and pos that name no pair or row: zero rows, and terms that are left out."""
    T, k, K = 6, 2, 24
    x, rows = normal((T, K), 1, dt), normal((T * k, K), 2, dt)
    src = ints([0, 11, 12, -1, (1 << 31) - 1, -(1 << 31), 5, 3, 3, 100, 1, 2])
    want = torch.stack([x[p // k] if 0 <= p < T * k else torch.zeros_like(x[0]) for p in src.tolist()])
    assert torch.equal(S.expert_gather(x, src), want)
    w = torch.zeros((1, 8, K), dtype=DT[dt], device=DEV) + 1
    o = offsets_of([T * k])
    assert torch.equal(S.grouped_fwd(x, w, w, o, src=src), S.grouped_fwd(want, w, w, o))
    pos = ints([[0, 12], [1, -1], [(1 << 31) - 1, 2], [-(1 << 31), 3], [4, 4], [5, 100]])
    y = S.expert_combine(rows, pos)
    for t, p in enumerate(pos.tolist()):
        live = [rows[r].float() for r in p if 0 <= r < T * k]
        assert torch.equal(y[t], sum(live, torch.zeros(K, device=DEV)).to(DT[dt])), t


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 8, 8), (97, 2, 5, 200, 264), (300, 4, 12, 136, 520), (40, 8, 64, 72, 264),
                                       (1300, 2, 40, 1040, 136)])
def test_gathered_rows_give_what_rows_give(T, k, E, N, K, dt):
    """With src the same bits as on rows gathered before."""
    g = np.random.default_rng(T)
    ids = g.integers(0, E, size=(T, k))
    ids[g.uniform(size=ids.shape) < 0.1] = -1
    offsets, src, pos = S.expert_plan(ints(ids).reshape(T, k), E)
    x, wg, wu = normal((T, K), 1, dt), normal((E, N, K), 2, dt, K ** -0.5), normal((E, N, K), 3, dt, K ** -0.5)
    rows = S.expert_gather(x, src)
    assert torch.equal(S.grouped_fwd(x, wg, wu, offsets, src=src), S.grouped_fwd(rows, wg, wu, offsets))
    dh = normal((T * k, N), 4, dt)
    ws = workspace(S.grouped_bwd_workspace_bytes(DT[dt], T * k, N, K, gathered=True))
    got = S.grouped_bwd(x, wg, wu, dh, offsets, src=src, workspace=ws)
    for a, b in zip(got, S.grouped_bwd(rows, wg, wu, dh, offsets)):
        assert torch.equal(a, b)
    only_x = S.grouped_bwd(x, wg, wu, dh, offsets, src=src, need_dw=False)
    only_w = S.grouped_bwd(x, wg, wu, dh, offsets, src=src, need_dx=False)
    assert only_x[1] is only_x[2] is only_w[0] is None
    assert torch.equal(only_x[0], got[0]) and torch.equal(only_w[1], got[1]) and torch.equal(only_w[2], got[2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_stacked_and_sliced_inputs(dt):
    """Halves of a stacked [E, 2N, K] are taken as they are; strided and misaligned tensors are copied."""
    counts, offsets, R = sizes("ragged")
    E, N, K = len(counts), 136, 72
    both = normal((E, 2 * N, K), 1, dt)
    wg, wu = both[:, :N], both[:, N:]
    wide = normal((R, K + 5), 2, dt)
    x = wide[:, 3:K + 3]
    dh = normal((N, R), 3, dt).t()
    h = S.grouped_fwd(x, wg, wu, offsets)
    assert torch.equal(h, S.grouped_fwd(x.contiguous(), wg.contiguous(), wu.contiguous(), offsets))
    for a, b in zip(S.grouped_bwd(x, wg, wu, dh, offsets),
                    S.grouped_bwd(x.contiguous(), wg.contiguous(), wu.contiguous(), dh.contiguous(), offsets)):
        assert torch.equal(a, b)
    flat = torch.empty(E * K * N + 1, dtype=DT[dt], device=DEV)
    wd = flat[1:].view(E, K, N).copy_(normal((E, K, N), 4, dt))
    for a, b in zip(S.grouped_mm_bwd(h, wd, x, offsets), S.grouped_mm_bwd(h, wd.clone(), x.contiguous(), offsets)):
        assert torch.equal(a, b)


def test_infinities_stay_with_their_expert():
    counts, offsets, R = sizes("tiles")
    E, N, K = len(counts), 72, 136
    x, w, dy = normal((R, K), 1, "bf16"), normal((E, N, K), 2, "bf16"), normal((R, N), 3, "bf16")
    y0, (dx0, dw0) = S.grouped_mm(x, w, offsets), S.grouped_mm_bwd(x, w, dy, offsets)
    a, b = int(offsets[2]), int(offsets[3])
    w2, x2, dy2 = w.clone(), x.clone(), dy.clone()
    w2[2, 5, 7], x2[a, 3], dy2[b - 1, 1] = math.inf, math.nan, math.inf
    y, (dx, dw) = S.grouped_mm(x2, w2, offsets), S.grouped_mm_bwd(x2, w2, dy2, offsets)
    rows = torch.ones(R, dtype=torch.bool, device=DEV)
    rows[a:b] = False
    assert torch.equal(y[rows], y0[rows]) and torch.equal(dx[rows], dx0[rows])
    others = [0, 1, 3, 4]
    assert torch.equal(dw[others], dw0[others])
    assert not torch.isfinite(y[a:b, 5]).any() and torch.isnan(y[a]).all()
    assert not torch.isfinite(dw[2, 1]).any() and torch.isnan(dw[2, :, 3]).all()


@pytest.mark.parametrize("N,K", [(0, 72), (72, 0)])
def test_empty_products(N, K):
    offsets = offsets_of([3, 4])
    x, w = torch.zeros((7, K), device=DEV), torch.zeros((2, N, K), device=DEV)
    y = S.grouped_mm(x, w, offsets, out=torch.full((7, N), math.nan, device=DEV))
    dx, dw = S.grouped_mm_bwd(x, w, torch.zeros((7, N), device=DEV), offsets,
                              out=(torch.full((7, K), math.nan, device=DEV), torch.zeros((2, N, K), device=DEV)))
    assert (y == 0).all() and (dx == 0).all()
    assert (S.grouped_fwd(x, w, w, offsets) == 0).all()
    for t in S.grouped_bwd(x, w, w, torch.zeros((7, N), device=DEV), offsets):
        assert (t == 0).all()
    # No rows at all: the weights' gradients are zero.
    none = torch.zeros((0, 72), device=DEV)
    wn = torch.ones((2, 8, 72), device=DEV)
    o = offsets_of([0, 0])
    assert S.grouped_mm(none, wn, o).shape == (0, 8)
    assert (S.grouped_mm_bwd(none, wn, torch.zeros((0, 8), device=DEV), o)[1] == 0).all()
    assert all((t == 0).all() for t in S.grouped_bwd(none, wn, wn, torch.zeros((0, 8), device=DEV), o)[1:])


# ------------------------------------------------------- the block as a whole

def oracle_block(x, wg, wu, wd, ids, w, dy, E, act):
    """(y, dx, dwg, dwu, dwd, dweights) in fp64."""
    offsets, src, pos = G.plan(ids, E)
    xr = G.gather(x, src, ids.shape[1])
    h, _ = G.gate_up(xr, wg, wu, offsets, act, 0.0)
    rows, _ = G.mm(h, wd, offsets, 0.0)
    y, _ = G.combine(rows, pos, w)
    drows, dw, _ = G.combine_bwd(dy, rows, pos, w)
    (dh, _), (dwd, _) = G.mm_bwd(h, wd, drows, offsets, 0.0)
    (dxr, _), (dwg, _), (dwu, _) = G.gate_up_bwd(xr, wg, wu, dh, offsets, act, 0.0)
    return y, G.combine(dxr, pos)[0], dwg, dwu, dwd, dw


def block_problem(dt, T=75, k=3, E=6, N=136, K=72, seed=5):
    logits = normal((T, E), seed, "f32")
    logits[3] = -math.inf
    logits[10, :4] = -math.inf
    ts = [normal((T, K), 1, dt), normal((E, N, K), 2, dt, K ** -0.5), normal((E, N, K), 3, dt, K ** -0.5),
          normal((E, K, N), 4, dt, N ** -0.5)]
    return [t.requires_grad_(True) for t in ts], logits.requires_grad_(True), normal((T, K), 6, dt), k


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_router_and_routed_mlp_train_together(dt, act):
    """Forward and every gradient, the router's logits among them, against the oracle: the whole is off by a few
    roundings of its type at each of its five stages, relative to the largest value (normwise 2e-2 and 2e-5)."""
    (x, wg, wu, wd), logits, dy, k = block_problem(dt)
    w, ids = S.router(logits, k)
    y = S.routed_mlp(x, wg, wu, wd, ids, w, act=act)
    got = torch.autograd.grad((y.float() * dy.float()).sum(), (x, wg, wu, wd, logits))
    want = oracle_block(*map(host, (x, wg, wu, wd)), ids.cpu().numpy(), host(w), host(dy), wg.shape[0], act)
    dlogits = S.route_bwd(logits.detach(), ids, torch.from_numpy(want[5]).float().to(DEV))
    tol = 2e-2 if dt == "bf16" else 2e-5
    for t, v, name in zip((y, *got), (*want[:5], host(dlogits)), ("y", "dx", "dwg", "dwu", "dwd", "dlogits")):
        err = np.abs(host(t) - v).max() / np.abs(v).max()
        print(f"routed_mlp {dt} {act} {name}: {err:.2e}", flush=True)
        assert err <= tol, name
    assert (y[3] == 0).all() and (got[0][3] == 0).all()


def test_pieces_give_what_the_whole_gives():
    (x, wg, wu, wd), logits, dy, k = block_problem("f32")
    w, ids = S.router(logits, k)
    leaves = (x, wg, wu, wd, logits)
    whole = S.routed_mlp(x, wg, wu, wd, ids, w)
    gw = torch.autograd.grad((whole * dy).sum(), leaves, retain_graph=True)
    offsets, src, pos = S.expert_plan(ids, wg.shape[0])
    h = S.grouped_swiglu(S.expert_rows(x, src, pos), wg, wu, offsets)
    y = S.expert_sum(S.grouped_linear(h, wd, offsets), pos, w)
    assert torch.equal(y, whole)
    for a, b in zip(torch.autograd.grad((y * dy).sum(), leaves), gw):
        assert torch.equal(a, b)


def test_some_inputs_need_no_gradient():
    (x, wg, wu, wd), logits, dy, k = block_problem("bf16")
    w, ids = S.route(logits.detach(), k)
    full = torch.autograd.grad((S.routed_mlp(x, wg, wu, wd, ids, w.requires_grad_(True)) * dy).sum(), (x, wg, wu, wd, w))
    for i, keep in enumerate(((0,), (1,), (3,), (4,), (0, 4), (2, 3))):
        ts = [t.detach().requires_grad_(j in keep) for j, t in enumerate((x, wg, wu, wd, w))]
        got = torch.autograd.grad((S.routed_mlp(*ts[:4], ids, ts[4]) * dy).sum(), [ts[j] for j in keep])
        for a, j in zip(got, keep):
            assert torch.equal(a, full[j]), (i, j)


def test_matches_the_few_token_experts():
    """The same MLP as moe_fwd within both roundings (h there has 16 bits, here 8)."""
    T, E, N, K, k = 24, 8, 200, 264, 2
    x = normal((T, K), 1, "bf16")
    wg, wu, wd = normal((E, N, K), 2, "bf16", 0.05), normal((E, N, K), 3, "bf16", 0.05), normal((E, K, N), 4, "bf16", 0.05)
    w, ids = S.route(normal((T, E), 5, "f32"), k)
    a, b = S.moe_fwd(x, wg, wu, wd, ids, w).double(), S.routed_mlp(x, wg, wu, wd, ids, w).double()
    assert ((a - b).norm() / a.norm()).item() < 1e-2


def test_large_tokens_are_gathered_first(monkeypatch):
    """Tokens whose bytes pass 32 bits take the path over gathered rows (the limit is moved down here)."""
    import swiglu_mlp_fwd_amd.group_ops as ops
    (x, wg, wu, wd), logits, dy, k = block_problem("bf16")
    w, ids = S.route(logits.detach(), k)
    offsets, src, _ = S.expert_plan(ids, wg.shape[0])
    x, wg, wu = x.detach(), wg.detach(), wu.detach()
    want = S.grouped_fwd(x, wg, wu, offsets, src=src)
    monkeypatch.setattr(ops, "GATHER_BYTES", 64)
    assert torch.equal(S.grouped_fwd(x, wg, wu, offsets, src=src), want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_training_step_replays_in_a_graph(dt):
    """Router, routed MLP, gradients and clipping captured; every replay against the eager step, with eager work between
    replays, and with other routing from replay to replay."""
    (x, wg, wu, wd), logits, dy, k = block_problem(dt, T=130)
    leaves = (x, wg, wu, wd, logits)

    def step():
        w, ids = S.router(logits, k)
        y = S.routed_mlp(x, wg, wu, wd, ids, w)
        grads = torch.autograd.grad((y.float() * dy.float()).sum(), leaves)
        norm = S.clip_grads(grads, 0.5)
        return (y.detach(), norm, *grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    for rep in range(4):
        with torch.no_grad():
            logits.copy_(normal(logits.shape, 50 + rep, "f32"))
        eager = [t.detach().clone() for t in step()]
        torch.cuda.synchronize()
        for t in captured:
            t.detach().fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, eager)):
            assert torch.equal(a, b), f"replay {rep}, output {i}"
        S.expert_plan(torch.zeros((9000, 2), dtype=torch.int32, device=DEV), 7)
        torch.cuda.synchronize()


def test_on_a_side_stream_and_twice_at_once():
    """Two calls on two streams, a workspace each, give what one call gives."""
    counts, offsets, R = sizes("tiles")
    E, N, K = len(counts), 264, 328
    x, wg, wu, dh = normal((R, K), 1, "bf16"), normal((E, N, K), 2, "bf16", 0.05), normal((E, N, K), 3, "bf16", 0.05), normal((R, N), 4, "bf16")
    want = S.grouped_bwd(x, wg, wu, dh, offsets)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(S.grouped_bwd(x, wg, wu, dh, offsets))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ clipping

def grads_of(shapes, dts, seed=0, std=1.0):
    return [normal(s, seed + i, dt, std) for i, (s, dt) in enumerate(zip(shapes, dts))]


def check_clip(grads, limit, what, out=None):
    before = [host(g) for g in grads]
    norm, f = G.clip(before, limit)
    got = S.clip_grads(grads, limit, out=out)
    assert got.dtype == torch.float32 and got.shape == ()
    assert abs(got.item() - norm) <= 2 * U32 * norm, what
    for i, (t, b, g) in enumerate(zip(out if out is not None else grads, before, grads)):
        rnd = BF16_HALF_ULP if g.dtype == torch.bfloat16 else U32
        # The factor in fp32 and its product: a rounding each; below the normal range half of the least step.
        within(t, f * b, (2 * U32 + rnd) * 1.01 * np.abs(f * b) + 2.0 ** -134, f"{what} [{i}]")
        if out is not None:
            assert np.array_equal(host(g), b), f"{what}: gradient {i} changed"


@pytest.mark.parametrize("limit", [0.37, 1e9])
@pytest.mark.parametrize("into", [False, True])
def test_clip_of_many_kinds(limit, into):
    shapes = [(1,), (7, 3), (16384,), (16385,), (8191,), (8192,), (40000,), (0,), (3, 5, 7), (100001,), ()]
    dts = ["bf16", "f32", "bf16", "bf16", "f32", "f32", "f32", "f32", "bf16", "bf16", "f32"]
    grads = grads_of(shapes, dts)
    check_clip(grads, limit, f"clip {limit} {into}", [torch.full_like(g, math.nan) for g in grads] if into else None)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("count", [1, 191, 193, 320, 321, 700])
def test_clip_of_many_views_of_a_bucket(count, dt):
    """Views that start at any element, more than one launch's table, guards around the bucket."""
    g = np.random.default_rng(count)
    n = [int(v) for v in np.exp(g.uniform(0, 9, size=count))]
    b = guarded((sum(n) + 3,), DT[dt])
    b.t.copy_(normal((sum(n) + 3,), 1, dt))
    keep = b.t[-2:].clone()
    views = list(torch.split(b.t[1:1 + sum(n)], n))
    check_clip(views, 3.0, f"clip of {count} views {dt}")
    check_guards("clip", b)
    assert torch.equal(b.t[-2:], keep)
    o = guarded((sum(n) + 8,), DT[dt])
    outs = list(torch.split(o.t[5:5 + sum(n)], n))
    check_clip(views, 0.5, f"clip of {count} views {dt} into others", outs)
    check_guards("clip", o)
    assert torch.isnan(o.t[:5]).all() and torch.isnan(o.t[5 + sum(n):]).all()


def test_clip_extremes():
    big = torch.full((1000,), 3e38, device=DEV)
    assert S.grad_norm([big]).item() == math.inf                     # 9.5e39: past fp32, not past the sum
    small = torch.full((4,), 1e-38, device=DEV)
    assert abs(S.grad_norm([small]).item() / 2e-38 - 1) < 1e-6       # squares of 1e-76
    g = [torch.tensor([3.0, math.nan], device=DEV), torch.ones(3, device=DEV, dtype=torch.bfloat16)]
    assert math.isnan(S.clip_grads(g, 1.0).item()) and all(torch.isnan(t).all() for t in g)
    g = [torch.tensor([3.0, -math.inf], device=DEV), torch.ones(3, device=DEV)]
    assert S.clip_grads(g, 1.0).item() == math.inf
    assert g[0][0] == 0 and torch.isnan(g[0][1]) and (g[1] == 0).all()
    g = [torch.ones(5, device=DEV)]
    S.clip_grads(g, math.inf)
    assert (g[0] == 1).all()
    S.clip_grads(g, 0.0)
    assert (g[0] == 0).all()
    assert S.clip_grads([torch.zeros(9, device=DEV)], 1.0).item() == 0.0
    assert S.grad_norm([torch.zeros(0, device=DEV)]).item() == 0.0


def test_clip_of_strided_gradients():
    a = normal((12, 20), 1, "f32")
    for t in (a.t(), a[:, ::2], a[::3, 5:9]):
        before, rest = host(t), host(a)
        norm, f = G.clip([before, np.ones(4)], 2.0)
        other = torch.ones(4, device=DEV)
        got = S.clip_grads([t, other], 2.0)
        assert abs(got.item() - norm) <= 2 * U32 * norm
        within(t, f * before, 3 * U32 * np.abs(before), f"strided {tuple(t.stride())}")
        at = torch.zeros_like(a, dtype=torch.bool)
        at.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(True)
        untouched = ~at.cpu().numpy()
        assert np.array_equal(host(a)[untouched], rest[untouched])
    out = torch.empty((20, 12), device=DEV).t()
    g = normal((12, 20), 2, "f32")
    S.clip_grads([g], 1.0, out=[out])
    n, f = G.clip([host(g)], 1.0)
    within(out, f * host(g), 3 * U32 * np.abs(host(g)), "into a transposed tensor")


@pytest.mark.parametrize("dt,n", [("bf16", 97_000_003), ("f32", 48_000_001)])
def test_clip_of_many_bytes_into_out(dt, n):
    """Results past the caches, chunks that start and end inside their tensors' 16 bytes."""
    flat = normal((n,), 3, dt)
    g = [flat[:11], flat[11:n // 2], flat[n // 2:n - 5], flat[n - 5:]]
    keep, res = flat.clone(), torch.full((n + 8,), 7.0, dtype=DT[dt], device=DEV)
    out = [res[4:15], res[15:4 + n // 2], res[4 + n // 2:n - 1], res[n - 1:n + 4]]
    norm = S.clip_grads(g, 2.5, out=out)
    want = math.sqrt(sum(c.double().square().sum().item() for c in flat.split(1 << 24)))
    assert abs(norm.item() - want) <= 2 ** -23 * want
    for a, b in zip(flat.split(1 << 24), res[4:n + 4].split(1 << 24)):
        e = a.double() * (2.5 / (want + 1e-6))
        assert ((b.double() - e).abs() <= e.abs() * (torch.finfo(DT[dt]).eps / 2 + 2 ** -22)).all()
    assert torch.equal(flat, keep) and (res[:4] == 7).all() and (res[n + 4:] == 7).all()


def test_clip_of_inference_tensors():
    with torch.inference_mode():
        g = [torch.full((3,), 2.0, device=DEV), torch.zeros(2, device=DEV)]
        S.clip_grads(g, 1.0, eps=0.0)
    assert torch.allclose(g[0], torch.full((3,), 2 / math.sqrt(12), device=DEV) )


def test_clip_is_seen_by_autograd():
    p = torch.ones(4, device=DEV, requires_grad=True)
    q = p * 2
    loss = (q * q).sum()
    S.clip_grads([q.detach()], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
