"""PyTorch-facing wrappers of the routed block's entry points: the router, the
few-token experts and the norms around a block.

Argument marshalling only, as in ops.py: shapes, dtypes and devices are
checked before the library is called, inputs are made contiguous (stacked
expert weights are not copied: their experts may lie apart), outputs are
allocated with torch.empty, and the library is called on the current HIP
stream.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from ._lib import MAX_EXPERTS, MAX_TOPK, MOE_MAX_TOKENS, SWIGLU_SCORE_SIGMOID, SWIGLU_SCORE_SOFTMAX, check, lib
from .ops import _act_code, _check_out, _dtype_code, _on_gpu, _p, _same

# The current stream's handle: these calls take a few microseconds on the GPU,
# and torch.cuda.current_stream alone takes two on the host.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

_SCORE = {"softmax": SWIGLU_SCORE_SOFTMAX, "sigmoid": SWIGLU_SCORE_SIGMOID}


def _stream(t: torch.Tensor) -> int:
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _rows(t: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """t as a contiguous [rows, cols]."""
    if t.dim() == 2 and t.is_contiguous():
        return t
    return t.reshape(rows, cols).contiguous()


def _rows16(t: torch.Tensor, rows: int, cols: int) -> tuple[torch.Tensor, int]:
    """The same and its address, on a 16-byte boundary as the library takes logits: a slice that starts elsewhere is
    copied."""
    if t.dim() != 2 or not t.is_contiguous():
        t = t.reshape(rows, cols).contiguous()
    at = t.data_ptr()
    if at & 15:
        t = t.clone()
        at = t.data_ptr()
    return t, at


def _lead(t: torch.Tensor, lead, cols: int) -> torch.Tensor:
    """[rows, cols] back to [*lead, cols]."""
    return t if len(lead) == 1 else t.reshape(*lead, cols)


def _score_code(score: str) -> int:
    try:
        return _SCORE[score]
    except KeyError:
        raise ValueError(f"score must be one of {sorted(_SCORE)}, got {score!r}") from None


def _logit_sizes(logits: torch.Tensor, k: int) -> tuple[tuple, int, int]:
    """(leading shape, tokens, experts) of logits [..., E]."""
    if logits.dim() < 1:
        raise ValueError("logits must be [..., E]")
    lead, E = logits.shape[:-1], logits.shape[-1]
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"logits must have 1 to {MAX_EXPERTS} experts, got {E}")
    if not 1 <= k <= min(E, MAX_TOPK):
        raise ValueError(f"k must be in 1..{min(E, MAX_TOPK)}, got {k}")
    return lead, math.prod(lead), E


def route(logits: torch.Tensor, k: int, score: str = "softmax", renorm: bool = True, scale: float = 1.0, out=None):
    """The k best experts of each token and their weights.

    logits [..., E] fp32 or bf16 -> (weights fp32 [..., k], ids int32 [..., k]), the greatest logit first, equal
    ones in order of index.  score "softmax" or "sigmoid"; renorm divides by the sum over the chosen; scale
    multiplies the weights.  A logit of -inf masks its expert: where fewer than k are left, the id is -1 and the
    weight 0.  `out` may pass preallocated (weights [T, k], ids [T, k])."""
    dt, sc = _dtype_code(logits), _score_code(score)
    lead, T, E = _logit_sizes(logits, k)
    if out is not None:
        w, ids = out
        _check_out(w, "weights", (T, k), torch.float32, logits.device)
        _check_out(ids, "ids", (T, k), torch.int32, logits.device)
    _on_gpu(logits)
    l2, at = _rows16(logits, T, E)   # l2: the copy, if one was made, lives until the launch
    if out is None:
        w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    check("swiglu_route_fwd", lib().swiglu_route_fwd(sc, int(renorm), dt, T, E, k, at, float(scale), _p(w),
                                                     _p(ids), _stream(logits)))
    return _lead(w, lead, k), _lead(ids, lead, k)


def route_bwd(logits: torch.Tensor, ids: torch.Tensor, dweights: torch.Tensor, score: str = "softmax",
              renorm: bool = True, scale: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """dlogits [..., E] (dtype of logits) of L = sum(dweights * weights), with (weights, ids) = route(logits, ...);
    score, renorm and scale as given there.  `out` may pass a preallocated [T, E], on a 16-byte boundary."""
    dt, sc = _dtype_code(logits), _score_code(score)
    if ids.dim() < 1:
        raise ValueError("ids must be [..., k]")
    k = ids.shape[-1]
    lead, T, E = _logit_sizes(logits, k)
    if tuple(ids.shape) != (*lead, k) or tuple(dweights.shape) != (*lead, k):
        raise ValueError(f"ids and dweights must be {(*lead, k)}, got {tuple(ids.shape)}, {tuple(dweights.shape)}")
    if ids.dtype != torch.int32 or dweights.dtype != torch.float32:
        raise TypeError(f"ids must be int32 and dweights float32, got {ids.dtype}, {dweights.dtype}")
    if ids.device != logits.device or dweights.device != logits.device:
        raise ValueError("ids and dweights must be on the device of logits")
    if out is not None:
        _check_out(out, "out", (T, E), logits.dtype, logits.device)
    _on_gpu(logits)
    l2, at = _rows16(logits, T, E)
    i2, d2 = _rows(ids, T, k), _rows(dweights, T, k)
    d = out if out is not None else torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    check("swiglu_route_bwd", lib().swiglu_route_bwd(sc, int(renorm), dt, T, E, k, at, float(scale), _p(i2),
                                                     _p(d2), _p(d), _stream(logits)))
    return _lead(d, lead, E)


def moe_workspace_bytes(T: int, N: int, K: int, k: int) -> int:
    return int(lib().swiglu_moe_workspace_bytes(T, N, K, k))


def _expert_weights(t: torch.Tensor, rows: int, cols: int) -> tuple[torch.Tensor, int]:
    """Stacked [E, rows, cols] weights and the elements between experts; each
    expert dense, experts apart as the tensor has them (a slice of a stacked
    pair needs no copy)."""
    e, r, c = t.stride()
    one = t.shape[0] <= 1                        # its stride means nothing
    dense = (c == 1 or cols <= 1) and (r == cols or rows <= 1) and (one or (e >= rows * cols and e % 8 == 0))
    if not dense:
        t = t.contiguous()
        e = rows * cols
    return t, (rows * cols if one else e)


def moe_fwd(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, wd: torch.Tensor, ids: torch.Tensor,
            weights: torch.Tensor, act: str = "silu", workspace: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """The routed SwiGLU (act "silu") or GeGLU ("gelu_tanh") MLP for at most 64 tokens, bf16:

        y[t] = sum_j weights[t, j] * Wd_e (act(Wg_e x[t]) * (Wu_e x[t])),  e = ids[t, j].

    x [..., K]; wg, wu [E, N, K] and wd [E, K, N], whose experts may lie apart (w[:, :N] and w[:, N:] of a stacked
    [E, 2N, K] are taken as they are); ids int32 and weights fp32 [..., k], as route gives them (an id outside
    [0, E) is skipped).  Returns y [..., K].  `out` may pass a preallocated [T, K]; `workspace` a uint8 device
    buffer of at least moe_workspace_bytes(...) bytes (a smaller or missing one is replaced)."""
    _same(x, wg, wu, wd)
    if x.dtype != torch.bfloat16:
        raise TypeError("moe_fwd is bf16 only")
    lead, K = x.shape[:-1], x.shape[-1]
    T = math.prod(lead)
    if wg.dim() != 3:
        raise ValueError(f"wg must be [E, N, K], got {tuple(wg.shape)}")
    E, N = wg.shape[0], wg.shape[1]
    if wg.shape != (E, N, K) or wu.shape != (E, N, K) or wd.shape != (E, K, N):
        raise ValueError(f"weights must be [E, N, K], [E, N, K], [E, K, N] with K = {K}, got {tuple(wg.shape)}, "
                         f"{tuple(wu.shape)}, {tuple(wd.shape)}")
    if ids.dim() < 1 or ids.shape[:-1] != lead or ids.shape != weights.shape:
        raise ValueError(f"ids and weights must be {(*lead, 'k')}, got {tuple(ids.shape)}, {tuple(weights.shape)}")
    k = ids.shape[-1]
    if ids.dtype != torch.int32 or weights.dtype != torch.float32:
        raise TypeError(f"ids must be int32 and weights float32, got {ids.dtype}, {weights.dtype}")
    if ids.device != x.device or weights.device != x.device:
        raise ValueError("ids and weights must be on the device of x")
    if T > MOE_MAX_TOKENS:
        raise ValueError(f"moe_fwd takes at most {MOE_MAX_TOKENS} tokens, got {T}")
    if out is not None:
        _check_out(out, "out", (T, K), x.dtype, x.device)
    if workspace is not None and (workspace.device != x.device or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the device of x")
    _on_gpu(x)
    x2, i2, w2 = _rows(x, T, K), _rows(ids, T, k), _rows(weights, T, k)
    wg, sg = _expert_weights(wg, N, K)
    wu, su = _expert_weights(wu, N, K)
    wd, sd = _expert_weights(wd, K, N)
    need = int(lib().swiglu_moe_workspace_bytes(T, N, K, k))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    y = out if out is not None else torch.empty((T, K), dtype=x.dtype, device=x.device)
    check("swiglu_moe_fwd", lib().swiglu_moe_fwd(_act_code(act), T, E, k, N, K, _p(x2), _p(i2), _p(w2), _p(wg),
                                                 sg, _p(wu), su, _p(wd), sd, _p(y), _p(workspace),
                                                 workspace.numel() * workspace.element_size(), _stream(x)))
    return _lead(y, lead, K)


def _norm_sizes(like: torch.Tensor, w_out, gate, w_in) -> tuple[int, int, int]:
    """(rows, cols, groups) and the checks of the weights' shapes."""
    if like.dim() < 1:
        raise ValueError("the residual must be [..., cols]")
    cols = like.shape[-1]
    rows = math.prod(like.shape[:-1])
    for t, name in ((w_out, "w_out"), (w_in, "w_in")):
        if t is not None and t.shape != (cols,):
            raise ValueError(f"{name} must have shape {(cols,)}, got {tuple(t.shape)}")
    groups = 0
    if gate is not None:
        if gate.dim() not in (1, 2) or gate.shape[-1] != cols:
            raise ValueError(f"gate must be [{cols}] or [groups, {cols}], got {tuple(gate.shape)}")
        groups = gate.shape[0] if gate.dim() == 2 else 1
        if groups < 1 or rows % groups != 0:
            raise ValueError(f"gate has {groups} groups, which do not divide {rows} rows")
    return rows, cols, groups


def _contig(t):
    return t if t is None or t.is_contiguous() else t.contiguous()


def _like(t):
    """An output shaped as t (contiguous or None)."""
    return None if t is None else torch.empty_like(t)


def block_norm(res: torch.Tensor, y: torch.Tensor | None = None, w_out: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, w_in: torch.Tensor | None = None, skip: float = 1.0,
               scale: float = 1.0, w_offset: float = 0.0, eps: float = 1e-6, out=None):
    """The norms around a block in one pass, with RMS(v) = v / sqrt(mean(v^2) + eps) over the last dimension:

        n = RMS(y) * (w_offset + w_out)   (n = y without w_out)
        res_out = skip * res + scale * gate * n
        z = RMS(res_out) * (w_offset + w_in)

    res, y [..., cols]; w_out, w_in [cols]; gate [cols] or [groups, cols], a row for each of `groups` equal runs of
    rows.  All fp32 or all bf16.  Returns (res_out, z), z None without w_in; without y there is no block to join:
    (None, RMS(res) * (w_offset + w_in)).  `out` may pass preallocated (res_out, z) (None where there is none)."""
    given = [t for t in (res, y, w_out, gate, w_in) if t is not None]
    _same(*given)
    dt = _dtype_code(res)
    if y is not None and y.shape != res.shape:
        raise ValueError(f"y must have the shape of res, {tuple(res.shape)}, got {tuple(y.shape)}")
    if y is None and (w_out is not None or gate is not None):
        raise ValueError("w_out and gate need y")
    if y is None and w_in is None:
        raise ValueError("block_norm needs y or w_in")
    rows, cols, groups = _norm_sizes(res, w_out, gate, w_in)
    if out is not None:
        ro, z = out
        if y is not None:
            _check_out(ro, "res_out", res.shape, res.dtype, res.device)
        if w_in is not None:
            _check_out(z, "z", res.shape, res.dtype, res.device)
        if (y is None and ro is not None) or (w_in is None and z is not None):
            raise ValueError("out has an output that this call does not compute")
    _on_gpu(res)
    res, y, w_out, gate, w_in = _contig(res), _contig(y), _contig(w_out), _contig(gate), _contig(w_in)
    if out is None:
        ro = _like(y)
        z = None if w_in is None else torch.empty_like(res)
    check("swiglu_block_norm_fwd", lib().swiglu_block_norm_fwd(
        dt, rows, cols, groups, _p(res), _p(y), _p(w_out), _p(gate), _p(w_in), float(skip), float(scale),
        float(w_offset), float(eps), _p(ro), _p(z), _stream(res)))
    return ro, z


def block_norm_bwd_workspace_bytes(rows: int, cols: int, groups: int = 0) -> int:
    """Bytes of workspace of block_norm_bwd; groups = 0 without a gate."""
    return int(lib().swiglu_block_norm_bwd_workspace_bytes(rows, cols, groups))


def block_norm_bwd(res_out: torch.Tensor | None, y: torch.Tensor | None = None, w_out: torch.Tensor | None = None,
                   gate: torch.Tensor | None = None, w_in: torch.Tensor | None = None,
                   dres_out: torch.Tensor | None = None, dz: torch.Tensor | None = None, skip: float = 1.0,
                   scale: float = 1.0, w_offset: float = 0.0, eps: float = 1e-6,
                   workspace: torch.Tensor | None = None, out=None):
    """Gradients of block_norm: (dres, dy, dw_out, dgate, dw_in), None for arguments that are None.

    res_out is block_norm's output (res itself where y is None; not needed without w_in); dres_out and dz the
    gradients of its outputs (dres_out None for 0, dz given exactly with w_in).  `out` may pass the five
    preallocated; `workspace` a uint8 device buffer of at least block_norm_bwd_workspace_bytes(...) bytes."""
    given = [t for t in (dz, dres_out, y, res_out, w_out, gate, w_in) if t is not None]
    if not given:
        raise ValueError("block_norm_bwd needs a gradient")
    _same(*given)
    like = given[0]
    dt = _dtype_code(like)
    if dz is None and dres_out is None:
        raise ValueError("block_norm_bwd needs dres_out or dz")
    if (dz is None) != (w_in is None):
        raise ValueError("dz must be given exactly where w_in is")
    if w_in is not None and res_out is None:
        raise ValueError("res_out is needed with w_in")
    if y is None and (w_out is not None or gate is not None or w_in is None):
        raise ValueError("w_out and gate need y, and without y there must be w_in")
    for t, name in ((y, "y"), (res_out, "res_out"), (dres_out, "dres_out"), (dz, "dz")):
        if t is not None and t.shape != like.shape:
            raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    rows, cols, groups = _norm_sizes(like, w_out, gate, w_in)
    if out is not None:
        if len(out) != 5:
            raise ValueError("out must be (dres, dy, dw_out, dgate, dw_in)")
        for t, of, name in zip(out, (like, y, w_out, gate, w_in), ("dres", "dy", "dw_out", "dgate", "dw_in")):
            if of is not None:
                _check_out(t, name, of.shape, like.dtype, like.device)
            elif t is not None:
                raise ValueError("out has an output that this call does not compute")
    if workspace is not None and (workspace.device != like.device or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the device of the inputs")
    _on_gpu(like)
    res_out, y, w_out, gate, w_in = _contig(res_out), _contig(y), _contig(w_out), _contig(gate), _contig(w_in)
    dres_out, dz = _contig(dres_out), _contig(dz)
    if out is None:
        out = (_like(dz if dz is not None else dres_out), _like(y), _like(w_out), _like(gate), _like(w_in))
    dres, dy, dw_out, dgate, dw_in = out
    need = int(lib().swiglu_block_norm_bwd_workspace_bytes(rows, cols, groups))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=like.device)
    check("swiglu_block_norm_bwd", lib().swiglu_block_norm_bwd(
        dt, rows, cols, groups, _p(res_out), _p(y), _p(w_out), _p(gate), _p(w_in), _p(dres_out), _p(dz), float(skip),
        float(scale), float(w_offset), float(eps), _p(dres), _p(dy), _p(dw_out), _p(dgate), _p(dw_in),
        _p(workspace), workspace.numel() * workspace.element_size(), _stream(like)))
    return dres, dy, dw_out, dgate, dw_in


class RouterFunction(torch.autograd.Function):
    """Autograd wrapper of route: gradients of the weights; ids have none.  The gradients have no derivative of their
    own (asking for one raises)."""

    @staticmethod
    def forward(ctx, logits, k, score="softmax", renorm=True, scale=1.0):
        w, ids = route(logits, k, score=score, renorm=renorm, scale=scale)
        ctx.save_for_backward(logits, ids)
        ctx.cfg = (score, renorm, scale)
        ctx.mark_non_differentiable(ids)
        return w, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, dw, _):
        logits, ids = ctx.saved_tensors
        score, renorm, scale = ctx.cfg
        return route_bwd(logits, ids, dw, score=score, renorm=renorm, scale=scale), None, None, None, None


def router(logits, k: int, score: str = "softmax", renorm: bool = True, scale: float = 1.0):
    """Differentiable route: (weights, ids)."""
    return RouterFunction.apply(logits, k, score, renorm, scale)


class BlockNormFunction(torch.autograd.Function):
    """Autograd wrapper of block_norm; the constants skip, scale, w_offset and eps are not trained.  The gradients have
    no derivative of their own (asking for one raises)."""

    @staticmethod
    def forward(ctx, res, y, w_out, gate, w_in, skip=1.0, scale=1.0, w_offset=0.0, eps=1e-6):
        ro, z = block_norm(res, y, w_out=w_out, gate=gate, w_in=w_in, skip=skip, scale=scale, w_offset=w_offset,
                           eps=eps)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(ro if y is not None else res, y, w_out, gate, w_in)
        ctx.cfg = dict(skip=skip, scale=scale, w_offset=w_offset, eps=eps)
        return ro, z

    @staticmethod
    @once_differentiable
    def backward(ctx, dro, dz):
        ro, y, w_out, gate, w_in = ctx.saved_tensors
        if w_in is not None and dz is None:
            dz = torch.zeros_like(ro)
        if dro is None and dz is None:
            return (None,) * 9
        dres, dy, dw_out, dgate, dw_in = block_norm_bwd(ro, y, w_out=w_out, gate=gate, w_in=w_in, dres_out=dro, dz=dz,
                                                        **ctx.cfg)
        return dres, dy, dw_out, dgate, dw_in, None, None, None, None


def block_norms(res, y=None, w_out=None, gate=None, w_in=None, skip: float = 1.0, scale: float = 1.0,
                w_offset: float = 0.0, eps: float = 1e-6):
    """Differentiable block_norm: (res_out, z)."""
    return BlockNormFunction.apply(res, y, w_out, gate, w_in, skip, scale, w_offset, eps)
