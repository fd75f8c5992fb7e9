"""The operators around the SwiGLU stage of a routed block: plain forms, exact values and the cases they are timed on.

Three operators (each case names its one in "op"):

  route_fwd, route_bwd   the router: the k best experts of each token's logits and their weights, and its gradient
  moe                    the routed SwiGLU MLP for a few tokens: each token's experts, weighted and added
  norm_fwd, norm_bwd     the norms around a block: RMSNorm of its output, gate, residual scale, and the next block's
                         RMSNorm, in one pass, and its gradients

`run` computes them in elementary torch operations in fp32, rounded once at the end, or, where `own` is true, through
the package's entry points.  `exact` computes them from the definitions in fp64.
"""
import math

import torch

own = False
DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # A call that is all latency: three tokens, a small odd problem, GeGLU, one slot dropped by capacity.
        dict(name="moe_small_odd", op="moe", T=3, E=5, k=2, N=200, K=264, act="gelu_tanh", dropped=True),
        # Decoding one sequence: two of eight experts of the benchmark's decode shape.
        dict(name="moe_one_token", op="moe", T=1, E=8, k=2, N=6912, K=1536, act="silu", dropped=False),
        # Decoding eight sequences on the wide decode shape: nearly every expert is read.
        dict(name="moe_wide_8", op="moe", T=8, E=8, k=2, N=11008, K=4096, act="silu", dropped=False),
        # Decoding 64 sequences with many small experts: about eight tokens for each expert.
        dict(name="moe_fine_64", op="moe", T=64, E=64, k=8, N=1024, K=2048, act="silu", dropped=False),
        # The router of a decoding batch.
        dict(name="route_decode", op="route_fwd", T=8, E=64, k=8, dtype="bf16", score="softmax", renorm=True,
             scale=1.0, masked=False),
        # The router of a training batch.
        dict(name="route_train", op="route_fwd", T=32768, E=128, k=8, dtype="f32", score="softmax", renorm=True,
             scale=1.0, masked=False),
        # Sigmoid scores, an expert count that is no power of two, masked experts, padding rows with none left.
        dict(name="route_masked_odd", op="route_fwd", T=4001, E=60, k=4, dtype="bf16", score="sigmoid", renorm=True,
             scale=2.5, masked=True),
        # The router's gradient of a training batch: dense, since the softmax is over all experts.
        dict(name="route_bwd_train", op="route_bwd", T=32768, E=128, k=8, dtype="f32", score="softmax", renorm=False,
             scale=1.0, masked=False),
        # Between two blocks while decoding eight sequences.
        dict(name="norm_decode", op="norm_fwd", rows=8, cols=4096, dtype="bf16", has_y=True, post=True, groups=0,
             pre=True, skip=1.0, scale=1.0, w_offset=0.0),
        # Between two blocks of a training batch, with a gate for each channel.
        dict(name="norm_train", op="norm_fwd", rows=8192, cols=4096, dtype="bf16", has_y=True, post=True, groups=1,
             pre=True, skip=1.0, scale=0.5, w_offset=0.0),
        # The gradients of the same.
        dict(name="norm_bwd_train", op="norm_bwd", rows=8192, cols=4096, dtype="bf16", has_y=True, post=True,
             groups=1, pre=True, skip=1.0, scale=0.5, w_offset=0.0),
        # fp32, odd sizes, three samples with a gate each, weights held as offsets from one.
        dict(name="norm_bwd_odd", op="norm_bwd", rows=1203, cols=2051, dtype="f32", has_y=True, post=True, groups=3,
             pre=True, skip=0.9, scale=1.5, w_offset=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, units):
    """An odd multiple of one of `units` in [lo, hi], spread over the logarithm (lo itself where none fits)."""
    unit = rng.choice([u for u in units if u <= hi])
    n = (_log_int(rng, lo, hi) // unit - 1) | 1
    return max(lo, n * unit)


def draw(rng):
    op = rng.choice(["moe", "moe", "route_fwd", "route_bwd", "norm_fwd", "norm_bwd"])
    if op == "moe":
        E = _log_int(rng, 4, 64)
        N, K = _size(rng, 128, 11008, (8, 16, 64)), _size(rng, 256, 4096, (8, 16, 64))
        while 6 * E * N * K > 1.6e9:            # bytes of every expert's weights; the widest listed case has 2.2e9
            E, N = max(4, E // 2), max(128, N // 16 * 8)
        return dict(op=op, T=_log_int(rng, 1, 64), E=E, k=rng.randint(1, min(8, E)), N=N, K=K,
                    act=rng.choice(["silu", "gelu_tanh"]), dropped=rng.random() < 0.3)
    if op.startswith("route"):
        E, renorm = _size(rng, 8, 512, (1, 4, 16)), rng.random() < 0.5
        # One renormalised choice has the constant weight `scale` and no gradient: at least two.
        return dict(op=op, T=_size(rng, 1, 4194304 // E, (1, 2)), E=E, k=rng.randint(2 if renorm else 1, 8),
                    dtype=rng.choice(["bf16", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=renorm, scale=rng.choice([1.0, 2.5]), masked=rng.random() < 0.4)
    groups = rng.choice([0, 1, 2, 4])
    cols = _size(rng, 64, 8192, (1, 8, 16, 64))
    per = max(1, _size(rng, 1, min(8192, 33554432 // cols), (1, 2)) // max(groups, 1))
    has_y = rng.random() < 0.8
    pre = (not has_y) or rng.random() < 0.7
    return dict(op=op, rows=per * max(groups, 1), cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]), has_y=has_y,
                post=has_y and rng.random() < 0.7, groups=groups if has_y else 0, pre=pre,
                skip=rng.choice([1.0, 0.9]), scale=rng.choice([1.0, 0.5, 1.5]), w_offset=rng.choice([0.0, 1.0]))


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.float32):
    t = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    return t if std == 1.0 else t.mul_(std)


def _pick(logits, k):
    """The k best of each row, ties to the lowest index, -1 for an expert masked by -inf."""
    v, i = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    return torch.where(v[:, :k] == -math.inf, -1, i[:, :k]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "moe":
        T, E, k, N, K = (case[v] for v in ("T", "E", "k", "N", "K"))
        s = dict(case=case, x=_normal(g, (T, K), dtype=torch.bfloat16),
                 wg=_normal(g, (E, N, K), 0.02, torch.bfloat16), wu=_normal(g, (E, N, K), 0.02, torch.bfloat16),
                 wd=_normal(g, (E, K, N), 0.02, torch.bfloat16))
        logits = _normal(g, (T, E))
        s["ids"] = _pick(logits, k)
        w = torch.gather(torch.softmax(logits, -1), 1, s["ids"].long())
        s["weights"] = (w / w.sum(-1, keepdim=True)).contiguous()
        if case["dropped"]:                     # the last choice of every second token found its expert full
            s["ids"][::2, k - 1] = -1
        s["y"] = torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
        if own:
            import swiglu_mlp_fwd_amd as S
            s["ws"] = torch.empty(S.moe_workspace_bytes(T, N, K, k), dtype=torch.uint8, device=DEV)
        return s
    if op.startswith("route"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = _normal(g, (T, E), 1.5)
        if case["masked"]:                      # experts out of use for some tokens; about 1 % padding rows
            u = torch.rand((T, E), generator=g, device=DEV)
            p = torch.rand((T, 1), generator=g, device=DEV)
            logits = torch.where((u < 0.2) | (p < 0.01), -math.inf, logits)
        logits = logits.to(_DT[case["dtype"]])
        s = dict(case=case, logits=logits)
        if op == "route_fwd":                   # a loop keeps its output buffers
            s["out"] = (torch.empty((T, k), dtype=torch.float32, device=DEV),
                        torch.empty((T, k), dtype=torch.int32, device=DEV))
        else:
            s["ids"] = _pick(logits, k)
            s["dweights"] = _normal(g, (T, k))
            s["out"] = torch.empty_like(logits)
        return s
    rows, cols, dt = case["rows"], case["cols"], _DT[case["dtype"]]

    def weight():
        return (_normal(g, (cols,), 0.1) + (1.0 - case["w_offset"])).to(dt)

    s = dict(case=case, res=_normal(g, (rows, cols), 1.0, dt),
             y=_normal(g, (rows, cols), 2.0, dt) if case["has_y"] else None,
             w_out=weight() if case["post"] else None, w_in=weight() if case["pre"] else None,
             gate=_normal(g, (case["groups"], cols), 0.5, dt) if case["groups"] else None)
    if op == "norm_bwd":
        s["dres_out"] = _normal(g, (rows, cols), 0.01, dt)
        s["dz"] = _normal(g, (rows, cols), 0.01, dt) if case["pre"] else None
        if own:
            import swiglu_mlp_fwd_amd as S
            s["ws"] = torch.empty(S.block_norm_bwd_workspace_bytes(rows, cols, case["groups"]), dtype=torch.uint8,
                                  device=DEV)
    return s


# ------------------------------------------------------------------- run

def run(state):
    if own:
        table = dict(moe=_own_moe, route_fwd=_own_route, route_bwd=_own_route_bwd, norm_fwd=_own_norm,
                     norm_bwd=_own_norm_bwd)
    else:
        table = dict(moe=_plain_moe, route_fwd=_plain_route, route_bwd=_plain_route_bwd, norm_fwd=_plain_norm,
                     norm_bwd=_plain_norm_bwd)
    return table[state["case"]["op"]](state)


# ---- the package's entry points

def _own_moe(s):
    import swiglu_mlp_fwd_amd as S
    return S.moe_fwd(s["x"], s["wg"], s["wu"], s["wd"], s["ids"], s["weights"], act=s["case"]["act"],
                     workspace=s["ws"], out=s["y"])


def _own_route(s):
    import swiglu_mlp_fwd_amd as S
    c = s["case"]
    return S.route(s["logits"], c["k"], score=c["score"], renorm=c["renorm"], scale=c["scale"], out=s["out"])


def _own_route_bwd(s):
    import swiglu_mlp_fwd_amd as S
    c = s["case"]
    return S.route_bwd(s["logits"], s["ids"], s["dweights"], score=c["score"], renorm=c["renorm"], scale=c["scale"],
                       out=s["out"])


def _present(*ts):
    return tuple(t for t in ts if t is not None)


def _own_norm(s):
    import swiglu_mlp_fwd_amd as S
    c = s["case"]
    return _present(*S.block_norm(s["res"], s["y"], w_out=s["w_out"], gate=s["gate"], w_in=s["w_in"], skip=c["skip"],
                                  scale=c["scale"], w_offset=c["w_offset"], eps=EPS))


def _own_norm_bwd(s):
    import swiglu_mlp_fwd_amd as S
    c = s["case"]
    return _present(*S.block_norm_bwd(s["res"], s["y"], w_out=s["w_out"], gate=s["gate"], w_in=s["w_in"],
                                      dres_out=s["dres_out"], dz=s["dz"], skip=c["skip"], scale=c["scale"],
                                      w_offset=c["w_offset"], eps=EPS, workspace=s["ws"]))


# ---- plain forms

def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    t = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return z / (1.0 + torch.exp(-2.0 * t))


def _plain_moe(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x, ids = s["x"].float(), s["ids"].long()
    w = torch.where(ids >= 0, s["weights"], 0.0)
    ids = ids.clamp(min=0)
    if T * k <= E:                              # few pairs: take each pair's weights out
        p = ids.reshape(-1)
        xp = x.repeat_interleave(k, 0).unsqueeze(-1)
        h = _act(torch.bmm(s["wg"][p].float(), xp), c["act"]) * torch.bmm(s["wu"][p].float(), xp)
        y = torch.bmm(s["wd"][p].float(), h).reshape(T, k, -1)
        return (y * w.unsqueeze(-1)).sum(1).to(torch.bfloat16)
    dense = torch.zeros((T, E), device=x.device).scatter_add_(1, ids, w)
    y = torch.zeros_like(x)
    for e in range(E):                          # every expert on every token, weighted by the router's weight or 0
        h = _act(x @ s["wg"][e].float().t(), c["act"]) * (x @ s["wu"][e].float().t())
        y += dense[:, e:e + 1] * (h @ s["wd"][e].float().t())
    return y.to(torch.bfloat16)


def _plain_route(s):
    c = s["case"]
    k = c["k"]
    l = s["logits"].float()
    left = l.clone()
    at = torch.arange(l.shape[1], device=l.device)
    ids = []
    for _ in range(k):                          # the greatest, the first of its equals; then without it
        m = left.max(-1, keepdim=True).values
        i = torch.where(left == m, at, l.shape[1]).min(-1, keepdim=True).values
        ids.append(torch.where(m == -math.inf, -1, i))
        left = torch.where(at == i, -math.inf, left)
    ids = torch.cat(ids, 1)
    lk = torch.where(ids >= 0, torch.gather(l, 1, ids.clamp(min=0)), -math.inf)
    top = lk[:, :1].clamp(min=torch.finfo(torch.float32).min)
    if c["score"] == "softmax":
        w = torch.exp(lk - top)
        z = w.sum(-1, keepdim=True) if c["renorm"] else torch.exp(l - top).sum(-1, keepdim=True)
    else:                                       # renormalised: sigmoid(l) e^-t, t = min(top, 0), keeps tiny scores
        t = top.clamp(max=0.0) if c["renorm"] else 0.0
        w = torch.where(lk > 0, 1.0 / (1.0 + torch.exp(-lk)), torch.exp(lk - t) / (1.0 + torch.exp(lk)))
        z = w.sum(-1, keepdim=True) if c["renorm"] else torch.ones_like(top)
    return c["scale"] * w / torch.where(z > 0, z, 1.0), ids.to(torch.int32)


def _plain_route_bwd(s):
    c = s["case"]
    l, ids = s["logits"].float(), s["ids"].long()
    dw = torch.where(ids >= 0, s["dweights"], 0.0) * c["scale"]
    at = ids.clamp(min=0)
    lk = torch.where(ids >= 0, torch.gather(l, 1, at), -math.inf)
    top = lk[:, :1].clamp(min=torch.finfo(torch.float32).min)
    dense = torch.zeros_like(l)
    if c["score"] == "softmax":
        pk = torch.exp(lk - top)
        p = torch.exp(l - top)
        z = (pk if c["renorm"] else p).sum(-1, keepdim=True)
        z = torch.where(z > 0, z, 1.0)
        pk, p = pk / z, p / z
        m = (pk * dw).sum(-1, keepdim=True)
        if c["renorm"]:
            return dense.scatter_add_(1, at, pk * (dw - m) * (ids >= 0)).to(s["logits"].dtype)
        return (p * (dense.scatter_add_(1, at, dw) - m)).to(s["logits"].dtype)
    sk = 1.0 / (1.0 + torch.exp(-lk))
    ck = 1.0 / (1.0 + torch.exp(lk))            # 1 - sigmoid
    if c["renorm"]:
        t = top.clamp(max=0.0)
        w = torch.where(lk > 0, sk, torch.exp(lk - t) * ck)
        z = w.sum(-1, keepdim=True)
        w = w / torch.where(z > 0, z, 1.0)
        d = w * (dw - (w * dw).sum(-1, keepdim=True)) * ck
    else:
        d = dw * sk * ck
    return dense.scatter_add_(1, at, torch.where(ids >= 0, d, 0.0)).to(s["logits"].dtype)


def _rstd(v):
    return 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def _rows_of_gate(gate, rows):
    """[groups, cols] -> [rows, cols]: rows of one sample lie together."""
    return gate.float().repeat_interleave(rows // gate.shape[0], 0)


def _plain_norm(s):
    c = s["case"]
    dt = s["res"].dtype
    r, out = s["res"].float(), []
    if s["y"] is not None:
        n = s["y"].float()
        if s["w_out"] is not None:
            n = n * _rstd(n) * (s["w_out"].float() + c["w_offset"])
        if s["gate"] is not None:
            n = n * _rows_of_gate(s["gate"], c["rows"])
        r = c["skip"] * r + c["scale"] * n
        out.append(r.to(dt))
    if s["w_in"] is not None:
        out.append((r * _rstd(r) * (s["w_in"].float() + c["w_offset"])).to(dt))
    return tuple(out)


def _norm_grad(v, r, d):
    """d(sum d * v * rstd(v)) / dv, with r = rstd(v)."""
    return r * d - v * (r * r * r * (d * v).mean(-1, keepdim=True))


def _plain_norm_bwd(s):
    c = s["case"]
    dt, rows, cols = s["res"].dtype, c["rows"], c["cols"]
    total = s["dres_out"].float()
    dw_in = dy = dw_out = dgate = None
    if s["w_in"] is not None:
        r, dz = s["res"].float(), s["dz"].float()
        k = _rstd(r)
        total = total + _norm_grad(r, k, dz * (s["w_in"].float() + c["w_offset"]))
        dw_in = (dz * r * k).sum(0).to(dt)
    if s["y"] is None:
        return _present(total.to(dt), dw_in)
    y = s["y"].float()
    k = _rstd(y) if s["w_out"] is not None else None
    w = s["w_out"].float() + c["w_offset"] if s["w_out"] is not None else None
    dn = c["scale"] * total
    if s["gate"] is not None:
        n = y if w is None else y * k * w
        dgate = (dn * n).reshape(c["groups"], rows // c["groups"], cols).sum(1).to(dt)
        dn = dn * _rows_of_gate(s["gate"], rows)
    if w is not None:
        dw_out = (dn * y * k).sum(0).to(dt)
        dn = _norm_grad(y, k, dn * w)
    return _present((c["skip"] * total).to(dt), dn.to(dt), dw_out, dgate, dw_in)


# ------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    return dict(moe=_exact_moe, route_fwd=_exact_route, route_bwd=_exact_route_bwd, norm_fwd=_exact_norm,
                norm_bwd=_exact_norm_bwd)[case["op"]](s)


def _exact_moe(s):
    act = s["case"]["act"]
    x, ids, w = s["x"].double(), s["ids"].tolist(), s["weights"].double()
    y = torch.zeros_like(x)
    for e in sorted({e for row in ids for e in row if e >= 0}):
        pairs = [(t, j) for t, row in enumerate(ids) for j, i in enumerate(row) if i == e]
        at = torch.tensor([t for t, _ in pairs], device=x.device)
        g = torch.matmul(s["wg"][e].double(), x[at].t())
        u = torch.matmul(s["wu"][e].double(), x[at].t())
        if act == "silu":
            h = g * torch.sigmoid(g) * u
        else:
            h = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))) * u
        o = torch.matmul(s["wd"][e].double(), h)
        for col, (t, j) in enumerate(pairs):
            y[t] += w[t, j] * o[:, col]
    return y


def _route64(l, ids, score, renorm, scale):
    """Weights of the chosen experts, differentiable in l (fp64); 0 where ids is -1."""
    gone = ids < 0
    if score == "softmax":
        logs = torch.gather(l, 1, ids.clamp(min=0))
        over = torch.where(gone, -math.inf, logs) if renorm else l
    else:
        logs = torch.nn.functional.logsigmoid(torch.gather(l, 1, ids.clamp(min=0)))
        over = torch.where(gone, -math.inf, logs) if renorm else torch.zeros_like(logs[:, :1])
    # A row with no expert left has no sum; its weights are 0 by definition.
    empty = gone.all(-1, keepdim=True)
    z = torch.logsumexp(torch.where(empty, 0.0, over), -1, keepdim=True)
    return scale * torch.where(gone, 0.0, torch.exp(torch.where(gone, 0.0, logs) - z))


def _exact_route(s):
    c = s["case"]
    l = s["logits"].double()
    order = torch.sort(-l, dim=-1, stable=True).indices[:, :c["k"]]
    ids = torch.where(torch.gather(l, 1, order) == -math.inf, -1, order)
    return _route64(l, ids, c["score"], c["renorm"], c["scale"]), ids.to(torch.int32)


def _exact_route_bwd(s):
    c = s["case"]
    real = s["logits"] != -math.inf             # -inf has no gradient: stand in a value that adds nothing
    l = torch.where(real, s["logits"].double(), -1e4).requires_grad_(True)
    ids = s["ids"].long()
    w = _route64(l, ids, c["score"], c["renorm"], c["scale"])
    (d,) = torch.autograd.grad((w * s["dweights"].double()).sum(), l)
    return torch.where(real, d, 0.0)


def _rms64(v):
    return v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)


def _update64(s, y, w_out, gate):
    c = s["case"]
    n = y if w_out is None else _rms64(y) * (w_out + c["w_offset"])
    if gate is not None:
        n = (n.reshape(c["groups"], -1, c["cols"]) * gate.unsqueeze(1)).reshape(n.shape)
    return c["scale"] * n


def _d(t):
    return None if t is None else t.double()


def _exact_norm(s):
    c = s["case"]
    r, out = s["res"].double(), []
    if s["y"] is not None:
        r = c["skip"] * r + _update64(s, s["y"].double(), _d(s["w_out"]), _d(s["gate"]))
        out.append(r)
    if s["w_in"] is not None:
        out.append(_rms64(r) * (s["w_in"].double() + c["w_offset"]))
    return tuple(out)


def _exact_norm_bwd(s):
    c = s["case"]
    total, dw_in = s["dres_out"].double(), None
    if s["w_in"] is not None:
        r = s["res"].double().requires_grad_(True)
        w = s["w_in"].double().requires_grad_(True)
        dr, dw_in = torch.autograd.grad((_rms64(r) * (w + c["w_offset"]) * s["dz"].double()).sum(), (r, w))
        total = total + dr
    if s["y"] is None:
        return _present(total, dw_in)
    ins = {n: s[n].double().requires_grad_(True) for n in ("y", "w_out", "gate") if s[n] is not None}
    up = _update64(s, ins["y"], ins.get("w_out"), ins.get("gate"))
    grads = dict(zip(ins, torch.autograd.grad((up * total).sum(), list(ins.values()))))
    return _present(c["skip"] * total, grads["y"], grads.get("w_out"), grads.get("gate"), dw_in)


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "moe":
        T, E, k, N, K = (case[v] for v in ("T", "E", "k", "N", "K"))
        read = E * (1.0 - (1.0 - k / E) ** T)   # experts that T tokens touch, on average
        return {"bytes": 6.0 * read * N * K + 4.0 * T * K + 8.0 * T * k, "flops": 6.0 * T * k * N * K}
    if op.startswith("route"):
        T, E, k = case["T"], case["E"], case["k"]
        b = 2 if case["dtype"] == "bf16" else 4
        if op == "route_fwd":
            return {"bytes": T * (b * E + 8.0 * k), "flops": 4.0 * T * E}
        return {"bytes": T * (2.0 * b * E + 8.0 * k), "flops": 6.0 * T * E}
    rows, cols = case["rows"], case["cols"]
    b = 2 if case["dtype"] == "bf16" else 4
    y, pre = int(case["has_y"]), int(case["pre"])
    vectors = int(case["post"]) + case["groups"] + pre
    if op == "norm_fwd":                        # in: res, y; out: res', z
        return {"bytes": b * cols * (rows * (1 + 2 * y + pre) + vectors), "flops": 12.0 * rows * cols}
    # in: dres', dz and res' where there is a second norm, y; out: dres, dy; and the weights' gradients
    return {"bytes": b * cols * (rows * (2 + 2 * pre + 2 * y) + 2 * vectors), "flops": 30.0 * rows * cols}
