"""The operators of a routed block that is trained or prefilled, over any number of tokens: plain forms, exact values
and the cases they are timed on.

Each case names its operator in "op"; R = T * k rows, one for each (token, choice) pair, lie in order of expert:

  plan                      the rows' order: offsets of each expert's rows, the pair of each row, the row of each pair
  combine_fwd, combine_bwd  each token's rows added with the router's weights, and the rows' and weights' gradients
  gate_up_fwd, gate_up_bwd  the gate/up stage h = act(x Wg_e^T) * (x Wu_e^T) of every row with its expert's weights,
                            the rows gathered from the tokens on the way, and its gradients
  product_fwd, product_bwd  y = x W_e^T of every row (the down projection), and its gradients
  clip                      the norm of all gradients together, and their clipping

A pair whose id is -1 was dropped; dropped pairs' rows come last, named by complements (~), and hold zeros.
`run` computes the operators in elementary torch operations in fp32, rounded once at the end, or, where `own` is true,
through the package's entry points.  `exact` computes them from the definitions in fp64.
"""
import math

import torch

own = False
DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The order of a decoding batch's rows: all latency.
        dict(name="plan_decode", op="plan", T=64, E=64, k=8, drop=0.0),
        # The order of a training batch's rows, a few tokens being padding.
        dict(name="plan_train", op="plan", T=32768, E=128, k=8, drop=0.02),
        # After the experts of a prefill: eight rows to a token.
        dict(name="combine_prefill", op="combine_fwd", T=4096, E=64, k=8, K=2048, dtype="bf16", drop=0.0),
        # Its gradient in training, two rows to a token, some over their expert's capacity.
        dict(name="combine_bwd_train", op="combine_bwd", T=8192, E=8, k=2, K=4096, dtype="bf16", drop=0.03),
        # A call that is all latency: small odd sizes, fp32, GeGLU, dropped pairs.
        dict(name="gate_up_small_odd", op="gate_up_fwd", T=97, E=5, k=2, N=200, K=264, dtype="f32", act="gelu_tanh",
             skew=0.5, drop=0.1),
        # A batch of 256 sequences, one token each, on many small experts: their weights are what there is to read.
        dict(name="gate_up_batch", op="gate_up_fwd", T=256, E=64, k=8, N=1024, K=2048, dtype="bf16", act="silu",
             skew=0.5, drop=0.0),
        # The benchmark's training shape with eight experts, two to a token.
        dict(name="gate_up_wide", op="gate_up_fwd", T=8192, E=8, k=2, N=14336, K=4096, dtype="bf16", act="silu",
             skew=0.3, drop=0.0),
        # Training many small experts: the gradients of the gate/up stage.
        dict(name="gate_up_bwd_fine", op="gate_up_bwd", T=4096, E=64, k=8, N=1024, K=2048, dtype="bf16", act="silu",
             skew=0.5, drop=0.0),
        # The down projection of the same.
        dict(name="product_fine", op="product_fwd", T=4096, E=64, k=8, N=2048, K=1024, dtype="bf16", skew=0.5,
             drop=0.0),
        # The down projection's gradients with few wide experts.
        dict(name="product_bwd_wide", op="product_bwd", T=8192, E=8, k=2, N=4096, K=11008, dtype="bf16", skew=0.3,
             drop=0.03),
        # All gradients of a model under the limit, as in most steps: many small fp32 tensors, views of one bucket.
        dict(name="clip_under", op="clip", n=420, least=1, most=400000, dtype="f32", over=False),
        # The gradients of four blocks of the benchmark's shape, over the limit, clipped into the optimizer's buffers.
        dict(name="clip_over", op="clip", n=24, least=4096, most=58720256, dtype="bf16", over=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, units):
    """An odd multiple of one of `units` in [lo, hi], spread over the logarithm (lo itself where none fits)."""
    unit = rng.choice([u for u in units if u <= hi])
    n = (_log_int(rng, lo, hi) // unit - 1) | 1
    return max(lo, n * unit)


def draw(rng):
    op = rng.choice(["plan", "combine_fwd", "combine_bwd", "gate_up_fwd", "gate_up_fwd", "gate_up_bwd", "gate_up_bwd",
                     "product_fwd", "product_fwd", "product_bwd", "clip"])
    if op == "clip":
        most = _log_int(rng, 1000, 20000000)
        return dict(op=op, n=_log_int(rng, 1, max(1, min(700, 700000000 // most))), least=rng.choice([1, 17, 256]),
                    most=most, dtype=rng.choice(["bf16", "f32"]), over=rng.random() < 0.6)
    E = _size(rng, 2, 256, (1, 2, 8))
    k = rng.randint(1, min(8, E))
    drop = rng.choice([0.0, 0.0, 0.1])
    if op == "plan":
        return dict(op=op, T=_size(rng, 1, 262144 // k, (1, 2)), E=E, k=k, drop=drop)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("combine"):
        K = _size(rng, 64, 8192, (8, 16, 64))
        return dict(op=op, T=_size(rng, 1, 33554432 // (k * K), (1, 2)), E=E, k=k, K=K, dtype=dtype, drop=drop)
    N, K = _size(rng, 128, 14336, (8, 16, 64)), _size(rng, 128, 8192, (8, 16, 64))
    while E * N * K > 4e8:                      # the experts' weights; the widest listed case has 4.7e8
        E, N = max(2, E // 2), max(128, N // 16 * 8)
    k = min(k, E)
    rows = min(200000000 // max(N, K), int(2.4e11 / (N * K)))
    c = dict(op=op, T=_size(rng, 1, max(1, rows // k), (1, 2)), E=E, k=k, N=N, K=K, dtype=dtype,
             skew=rng.choice([0.0, 0.3, 0.6]), drop=drop)
    if op.startswith("gate_up"):
        c["act"] = rng.choice(["silu", "gelu_tanh"])
    return c


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.float32):
    t = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    return t if std == 1.0 else t.mul_(std)


def _routing(g, T, E, k, skew, drop):
    """(weights, ids): the k best of E, some experts more liked than others, and dropped pairs (-1)."""
    logits = _normal(g, (T, E)) + skew * _normal(g, (1, E))
    w, ids = torch.topk(torch.softmax(logits, -1), k, dim=-1)
    if drop:
        gone = torch.rand((T, k), generator=g, device=DEV) < drop
        ids = torch.where(gone, -1, ids)
    return (w / w.sum(-1, keepdim=True)).contiguous(), ids.to(torch.int32).contiguous()


def _order(ids, E):
    """(offsets, src, pos) of pairs sorted by expert, the first pairs first, dropped ones last (as complements)."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat >= 0, flat, E)
    src = torch.sort(key, stable=True).indices
    pos = torch.empty_like(src)
    pos[src] = torch.arange(src.numel(), device=src.device)
    ends = torch.cumsum((key.unsqueeze(1) == torch.arange(E, device=key.device)).sum(0), 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    src = torch.where(flat[src] >= 0, src, ~src)
    pos = torch.where(flat >= 0, pos, ~pos)
    return offsets.to(torch.int32), src.to(torch.int32), pos.reshape(ids.shape).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "clip":
        return _prepare_clip(case, g)
    T, E, k = case["T"], case["E"], case["k"]
    w, ids = _routing(g, T, E, k, case.get("skew", 0.5), case["drop"])
    if case["op"] == "plan":
        return dict(case=case, ids=ids)
    s = dict(case=case)
    s["offsets"], s["src"], s["pos"] = _order(ids, E)
    dt, K, R = _DT[case["dtype"]], case["K"], T * k
    if case["op"].startswith("combine"):
        s.update(y=_normal(g, (R, K), 1.0, dt), weights=w)
        if case["op"] == "combine_bwd":
            s["dy"] = _normal(g, (T, K), 0.1, dt)
        return s
    N = case["N"]
    std = K ** -0.5
    if case["op"].startswith("gate_up"):
        s.update(x=_normal(g, (T, K), 1.0, dt), wg=_normal(g, (E, N, K), std, dt), wu=_normal(g, (E, N, K), std, dt))
        if case["op"] == "gate_up_bwd":
            s["dh"] = _normal(g, (R, N), 0.1, dt)
            if own:
                import swiglu_mlp_fwd_amd as S
                s["ws"] = torch.empty(S.grouped_bwd_workspace_bytes(dt, R, N, K, gathered=True), dtype=torch.uint8,
                                      device=DEV)
        return s
    s.update(x=_normal(g, (R, K), 1.0, dt), w=_normal(g, (E, N, K), std, dt))
    if case["op"] == "product_bwd":
        s["dy"] = _normal(g, (R, N), 0.1, dt)
    return s


def _sizes(case):
    """n sizes from least to most, spread over the logarithm."""
    n, lo, hi = case["n"], case["least"], case["most"]
    return [hi] if n == 1 else [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _prepare_clip(case, g):
    """Gradients of std about 0.01, views one after the other of a bucket, in an order of the seed's."""
    sizes = _sizes(case)
    sizes = [sizes[i] for i in torch.randperm(len(sizes), generator=g, device=DEV).tolist()]
    bucket = _normal(g, (sum(sizes),), 0.01, _DT[case["dtype"]])
    norm = 0.01 * math.sqrt(sum(sizes))
    s = dict(case=case, bucket=bucket, grads=list(torch.split(bucket, sizes)), limit=norm * (0.4 if case["over"] else 2.0))
    if case["over"]:
        s["bucket"] = torch.zeros_like(bucket)
        s["into"] = list(torch.split(s["bucket"], sizes))
    return s


# ------------------------------------------------------------------- run

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---- the package's entry points

def _own_plan(s):
    import swiglu_mlp_fwd_amd as S
    return S.expert_plan(s["ids"], s["case"]["E"])


def _own_combine(s):
    import swiglu_mlp_fwd_amd as S
    return S.expert_combine(s["y"], s["pos"], s["weights"])


def _own_combine_bwd(s):
    import swiglu_mlp_fwd_amd as S
    return S.expert_combine_bwd(s["dy"], s["y"], s["pos"], s["weights"])


def _own_gate_up(s):
    import swiglu_mlp_fwd_amd as S
    return S.grouped_fwd(s["x"], s["wg"], s["wu"], s["offsets"], src=s["src"], act=s["case"]["act"])


def _own_gate_up_bwd(s):
    import swiglu_mlp_fwd_amd as S
    return S.grouped_bwd(s["x"], s["wg"], s["wu"], s["dh"], s["offsets"], src=s["src"], act=s["case"]["act"],
                         workspace=s["ws"])


def _own_product(s):
    import swiglu_mlp_fwd_amd as S
    return S.grouped_mm(s["x"], s["w"], s["offsets"])


def _own_product_bwd(s):
    import swiglu_mlp_fwd_amd as S
    return S.grouped_mm_bwd(s["x"], s["w"], s["dy"], s["offsets"])


def _own_clip(s):
    import swiglu_mlp_fwd_amd as S
    return S.clip_grads(s["grads"], s["limit"], out=s.get("into")), s["bucket"]


_OWN = dict(plan=_own_plan, combine_fwd=_own_combine, combine_bwd=_own_combine_bwd, gate_up_fwd=_own_gate_up,
            gate_up_bwd=_own_gate_up_bwd, product_fwd=_own_product, product_bwd=_own_product_bwd, clip=_own_clip)


# ---- plain forms

def _plain_plan(s):
    return _order(s["ids"], s["case"]["E"])


def _plain_combine(s):
    rows = s["y"].float()[s["pos"].clamp(min=0).long()]          # [T, k, K]
    w = torch.where(s["pos"] >= 0, s["weights"], 0.0)
    return (rows * w.unsqueeze(-1)).sum(1).to(s["y"].dtype)


def _plain_combine_bwd(s):
    pos, dy = s["pos"], s["dy"].float().unsqueeze(1)
    live = pos >= 0
    at = torch.where(live, pos, ~pos).long()
    dw = torch.where(live, (s["y"].float()[at] * dy).sum(-1), 0.0)
    drows = torch.zeros_like(s["y"])
    drows[at.reshape(-1)] = (torch.where(live, s["weights"], 0.0).unsqueeze(-1) * dy).reshape(drows.shape).to(drows.dtype)
    return drows, dw


class _Padded:
    """Rows in order of expert as [E, C, cols], C the longest run, zeros behind the shorter ones; and back."""

    def __init__(self, offsets, R):
        first, count = offsets[:-1].long(), (offsets[1:] - offsets[:-1]).long()
        at = torch.arange(max(int(count.max()), 1), device=offsets.device)
        self.there = (at < count.unsqueeze(1)).unsqueeze(-1)                        # [E, C, 1]
        self.row = (first.unsqueeze(1) + at).clamp(max=max(R - 1, 0))               # [E, C]
        r = torch.arange(R, device=offsets.device)
        self.expert = torch.bucketize(r, offsets[1:].long(), right=True)
        self.live = (self.expert < first.numel()).unsqueeze(1)
        self.expert = self.expert.clamp(max=first.numel() - 1)
        self.slot = torch.where(self.live[:, 0], r - first[self.expert], 0)

    def pad(self, rows):
        return torch.where(self.there, rows[self.row].float(), 0.0)

    def back(self, padded, dtype):
        return torch.where(self.live, padded[self.expert, self.slot], 0.0).to(dtype)


def _token_rows(s):
    """Each row's token; a dropped pair's row is zero."""
    token = torch.where(s["src"] >= 0, s["src"], ~s["src"]).long() // s["case"]["k"]
    return torch.where(s["src"].unsqueeze(1) >= 0, s["x"][token], 0.0)


def _act_and_grad(z, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    t = 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    p = 1.0 / (1.0 + torch.exp(-t))
    dt = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z * z)
    return z * p, p + z * p * (1.0 - p) * dt


def _plain_gate_up(s):
    by = _Padded(s["offsets"], s["src"].numel())
    x = by.pad(_token_rows(s))
    g = torch.bmm(x, s["wg"].float().transpose(1, 2))
    u = torch.bmm(x, s["wu"].float().transpose(1, 2))
    return by.back(_act_and_grad(g, s["case"]["act"])[0] * u, s["x"].dtype)


def _plain_gate_up_bwd(s):
    dt = s["x"].dtype
    by = _Padded(s["offsets"], s["src"].numel())
    x, wg, wu, dh = by.pad(_token_rows(s)), s["wg"].float(), s["wu"].float(), by.pad(s["dh"])
    u = torch.bmm(x, wu.transpose(1, 2))
    a, da = _act_and_grad(torch.bmm(x, wg.transpose(1, 2)), s["case"]["act"])
    dg, du = dh * u * da, dh * a
    dx = by.back(torch.bmm(dg, wg) + torch.bmm(du, wu), dt)
    return dx, torch.bmm(dg.transpose(1, 2), x).to(dt), torch.bmm(du.transpose(1, 2), x).to(dt)


def _plain_product(s):
    by = _Padded(s["offsets"], s["x"].shape[0])
    return by.back(torch.bmm(by.pad(s["x"]), s["w"].float().transpose(1, 2)), s["x"].dtype)


def _plain_product_bwd(s):
    dt = s["x"].dtype
    by = _Padded(s["offsets"], s["x"].shape[0])
    x, dy = by.pad(s["x"]), by.pad(s["dy"])
    return by.back(torch.bmm(dy, s["w"].float()), dt), torch.bmm(dy.transpose(1, 2), x).to(dt)


def _plain_clip(s):
    squares = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]])
    norm = squares.sum().sqrt()
    factor = (s["limit"] / (norm + 1e-6)).clamp(max=1.0).float()
    if "into" in s:
        flat = torch.cat([t.float() * factor for t in s["grads"]])
        s["bucket"].copy_(flat)
    else:
        s["bucket"].copy_(s["bucket"].float() * factor)
    return norm.float(), s["bucket"]


_PLAIN = dict(plan=_plain_plan, combine_fwd=_plain_combine, combine_bwd=_plain_combine_bwd, gate_up_fwd=_plain_gate_up,
              gate_up_bwd=_plain_gate_up_bwd, product_fwd=_plain_product, product_bwd=_plain_product_bwd,
              clip=_plain_clip)


# ------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    return dict(plan=_exact_plan, combine_fwd=_exact_combine, combine_bwd=_exact_combine, gate_up_fwd=_exact_gate_up,
                gate_up_bwd=_exact_gate_up, product_fwd=_exact_product, product_bwd=_exact_product,
                clip=_exact_clip)[case["op"]](s)


def _exact_plan(s):
    ids, E = s["ids"].reshape(-1).tolist(), s["case"]["E"]
    rows = [[] for _ in range(E + 1)]
    for p, e in enumerate(ids):
        rows[e if e >= 0 else E].append(p)
    offsets, src, pos = [0], [], [0] * len(ids)
    for e, pairs in enumerate(rows):
        for p in pairs:
            pos[p] = len(src) if e < E else ~len(src)
            src.append(p if e < E else ~p)
        if e < E:
            offsets.append(len(src))

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)
    return ints(offsets), ints(src), ints(pos).reshape(s["ids"].shape)


def _exact_combine(s):
    c = s["case"]
    y = s["y"].double().requires_grad_(True)
    w = s["weights"].double().requires_grad_(True)
    out = torch.zeros((c["T"], c["K"]), dtype=torch.float64, device=DEV)
    for j in range(c["k"]):
        live = torch.nonzero(s["pos"][:, j] >= 0)[:, 0]
        out = out.index_add(0, live, w[live, j].unsqueeze(1) * y[s["pos"][live, j].long()])
    if c["op"] == "combine_fwd":
        return out.detach()
    return torch.autograd.grad((out * s["dy"].double()).sum(), (y, w))


def _runs(s):
    """(expert, first row, end) of the experts that have rows."""
    at = s["offsets"].tolist()
    return [(e, a, b) for e, (a, b) in enumerate(zip(at, at[1:])) if b > a]


def _exact_gate_up(s):
    c = s["case"]
    back = c["op"] == "gate_up_bwd"
    R, N, K = c["T"] * c["k"], c["N"], c["K"]
    src = s["src"].tolist()
    token = torch.tensor([p // c["k"] if p >= 0 else 0 for p in src], device=DEV)
    h = torch.zeros((R, N), dtype=torch.float64, device=DEV)
    dx = torch.zeros((R, K), dtype=torch.float64, device=DEV) if back else None
    dw = [torch.zeros((c["E"], N, K), dtype=torch.float64, device=DEV) for _ in range(2)] if back else None
    for e, a, b in _runs(s):
        leaf = [t.double().requires_grad_(back) for t in (s["x"][token[a:b]], s["wg"][e], s["wu"][e])]
        g, u = leaf[0] @ leaf[1].t(), leaf[0] @ leaf[2].t()
        if c["act"] == "silu":
            y = torch.nn.functional.silu(g) * u
        else:
            y = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))) * u
        if back:
            dx[a:b], dw[0][e], dw[1][e] = torch.autograd.grad((y * s["dh"][a:b].double()).sum(), leaf)
        else:
            h[a:b] = y
    return (dx, *dw) if back else h


def _exact_product(s):
    c = s["case"]
    R, N, K = c["T"] * c["k"], c["N"], c["K"]
    back = c["op"] == "product_bwd"
    y = torch.zeros((R, K if back else N), dtype=torch.float64, device=DEV)
    dw = torch.zeros((c["E"], N, K), dtype=torch.float64, device=DEV) if back else None
    for e, a, b in _runs(s):
        if back:
            y[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
            dw[e] = s["dy"][a:b].double().t() @ s["x"][a:b].double()
        else:
            y[a:b] = s["x"][a:b].double() @ s["w"][e].double().t()
    return (y, dw) if back else y


def _exact_clip(s):
    flat = torch.cat([t.double() for t in s["grads"]])
    norm = flat.norm()
    return norm, flat * min(1.0, s["limit"] / (norm.item() + 1e-6))


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "clip":
        b = 2 if case["dtype"] == "bf16" else 4
        n = sum(_sizes(case))
        return {"bytes": b * n * (2 if case["over"] else 1), "flops": (3.0 if case["over"] else 2.0) * n}
    T, E, k = case["T"], case["E"], case["k"]
    R = T * k
    if op == "plan":                            # in: ids; out: offsets, src, pos
        return {"bytes": 4.0 * (3 * R + E), "flops": 1.0 * R}
    b, K = 2 if case["dtype"] == "bf16" else 4, case["K"]
    live = R * (1.0 - case["drop"])
    if op == "combine_fwd":
        return {"bytes": b * K * (live + T) + 8.0 * R, "flops": 2.0 * live * K}
    if op == "combine_bwd":
        return {"bytes": b * K * (live + R + T) + 12.0 * R, "flops": 3.0 * live * K}
    N = case["N"]
    read = E * (1.0 - (1.0 - k * (1.0 - case["drop"]) / E) ** T)     # experts that have rows, on average
    if op == "gate_up_fwd":
        return {"bytes": b * (T * K + 2 * read * N * K + R * N) + 4.0 * R, "flops": 4.0 * live * N * K}
    if op == "gate_up_bwd":
        return {"bytes": b * (T * K + live * N + 2 * read * N * K + R * K + 2 * E * N * K) + 4.0 * R,
                "flops": 12.0 * live * N * K}
    if op == "product_fwd":
        return {"bytes": b * (live * K + read * N * K + R * N), "flops": 2.0 * live * N * K}
    return {"bytes": b * (live * (K + N) + read * N * K + R * K + E * N * K), "flops": 4.0 * live * N * K}
