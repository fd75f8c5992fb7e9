"""PyTorch-facing wrappers of the routed block's entry points for any number of
tokens: the order of rows by expert, the products grouped by expert, the sum of
a token's rows, their gradients, and the clipping of gradients.

Argument marshalling only, as in ops.py: shapes, dtypes and devices are checked
before the library is called, inputs are made contiguous and 16-byte aligned
(stacked expert weights are not copied: their experts may lie apart), outputs
are allocated with torch.empty, and the library is called on the current HIP
stream of the tensors' device.
"""
from __future__ import annotations

import itertools
import math
from array import array
from operator import attrgetter

import torch
from torch.autograd.function import once_differentiable

from ._lib import MAX_EXPERTS, MAX_TOPK, check, lib
from .block_ops import _expert_weights, _lead, _stream
from .ops import _DT, _act_code, _check_out, _dtype_code, _on_gpu, _p, _same

GATHER_BYTES = 1 << 31    # tokens of as many bytes are gathered before the products: row offsets are 32-bit there


def _call(name: str, like: torch.Tensor, *args) -> None:
    """The library's `name` on the current stream of the tensor's device, with that device current."""
    if like.get_device() == torch.cuda.current_device():
        check(name, getattr(lib(), name)(*args, _stream(like)))
    else:
        with torch.cuda.device(like.device):
            check(name, getattr(lib(), name)(*args, _stream(like)))


def _dense16(t: torch.Tensor) -> torch.Tensor:
    """t contiguous and on a 16-byte boundary."""
    if not t.is_contiguous():
        t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _weights16(t: torch.Tensor, rows: int, cols: int) -> tuple[torch.Tensor, int]:
    """Stacked expert weights and the elements between experts, the first on a 16-byte boundary."""
    t, stride = _expert_weights(t, rows, cols)
    if t.data_ptr() & 15:
        t, stride = t.contiguous().clone(), rows * cols
    return t, stride


def _check_offsets(offsets: torch.Tensor, E: int, device: torch.device) -> torch.Tensor:
    if offsets.shape != (E + 1,):
        raise ValueError(f"offsets must be [E + 1] = [{E + 1}], got {tuple(offsets.shape)}")
    if offsets.dtype != torch.int32:
        raise TypeError(f"offsets must be int32, got {offsets.dtype}")
    if offsets.device != device:
        raise ValueError(f"offsets must be on {device}, got {offsets.device}")
    return offsets.contiguous()


def _check_index(t: torch.Tensor, name: str, device: torch.device) -> None:
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _check_workspace(ws: torch.Tensor | None, device: torch.device) -> None:
    if ws is not None and (ws.device != device or not ws.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the device of the inputs")


def _workspace(ws: torch.Tensor | None, need: int, device: torch.device) -> tuple[torch.Tensor | None, int]:
    """A buffer of at least `need` bytes on a 256-byte boundary: the one given, or a new one."""
    if need == 0:
        return None, 0
    if ws is not None and ws.numel() * ws.element_size() >= need and ws.data_ptr() & 255 == 0:
        return ws, ws.numel() * ws.element_size()
    return torch.empty(need, dtype=torch.uint8, device=device), need


# --------------------------------------------------------- rows and tokens

def expert_plan_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(lib().swiglu_expert_plan_workspace_bytes(T, k, E))


def expert_plan(ids: torch.Tensor, E: int, workspace: torch.Tensor | None = None, out=None):
    """The order of all (token, choice) pairs by expert: (offsets int32 [E + 1], src int32 [T * k], pos as ids).

    ids int32 [..., k], as route gives them.  The rows of expert e are offsets[e] up to offsets[e + 1], in order of
    their pairs; src[r] is the pair t * k + j of row r and pos[..., j] the row of a pair.  Pairs whose id is outside
    [0, E) were dropped: their rows lie behind the last expert's, and src and pos name them by complements (~pair,
    ~row, negative).  `out` may pass preallocated (offsets, src, pos [T, k]); `workspace` a uint8 device buffer of
    expert_plan_workspace_bytes(T, k, E) bytes (a smaller or missing one is replaced)."""
    if ids.dim() < 1 or not 1 <= ids.shape[-1] <= MAX_TOPK:
        raise ValueError(f"ids must be [..., k] with k in 1..{MAX_TOPK}, got {tuple(ids.shape)}")
    if ids.dtype != torch.int32:
        raise TypeError(f"ids must be int32, got {ids.dtype}")
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"E must be in 1..{MAX_EXPERTS}, got {E}")
    lead, k = ids.shape[:-1], ids.shape[-1]
    T = math.prod(lead)
    dev = ids.device
    if out is not None:
        offsets, src, pos = out
        for t, name, shape in ((offsets, "offsets", (E + 1,)), (src, "src", (T * k,)), (pos, "pos", (T, k))):
            _check_out(t, name, shape, torch.int32, dev)
    _check_workspace(workspace, dev)
    _on_gpu(ids)
    ids = ids.contiguous()
    if out is None:
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        src = torch.empty(T * k, dtype=torch.int32, device=dev)
        pos = torch.empty((T, k), dtype=torch.int32, device=dev)
    ws, n = _workspace(workspace, int(lib().swiglu_expert_plan_workspace_bytes(T, k, E)), dev)
    _call("swiglu_expert_plan", ids, T, k, E, _p(ids), _p(offsets), _p(src), _p(pos), _p(ws), n)
    return offsets, src, _lead(pos, lead, k)


def _tokens_of(x: torch.Tensor, src: torch.Tensor) -> tuple[int, int, int]:
    """(T, k, K) of tokens x [..., K] and src [T * k]."""
    if x.dim() < 1 or src.dim() != 1:
        raise ValueError(f"x must be [..., K] and src [T * k], got {tuple(x.shape)}, {tuple(src.shape)}")
    _check_index(src, "src", x.device)
    T, K = math.prod(x.shape[:-1]), x.shape[-1]
    R = src.shape[0]
    if (T == 0 and R != 0) or (T > 0 and (R % T != 0 or not 1 <= R // T <= MAX_TOPK)):
        raise ValueError(f"src must have T * k elements, k in 1..{MAX_TOPK}: {R} of them for {T} tokens")
    return T, (R // T if T else 1), K


def expert_gather(x: torch.Tensor, src: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """rows[r] = x[src[r] // k], zeros where src[r] is negative: tokens x [..., K] as rows [T * k, K] in the order of
    expert_plan.  `out` may pass a preallocated [T * k, K]."""
    dt = _dtype_code(x)
    T, k, K = _tokens_of(x, src)
    if out is not None:
        _check_out(out, "out", (T * k, K), x.dtype, x.device)
    _on_gpu(x)
    x2, src = _dense16(x), src.contiguous()
    rows = out if out is not None else torch.empty((T * k, K), dtype=x.dtype, device=x.device)
    _call("swiglu_expert_gather", x, dt, T, k, K, _p(x2), _p(src), _p(rows))
    return rows


def _combine_sizes(rows: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor | None) -> tuple[tuple, int, int, int]:
    if pos.dim() < 1 or not 1 <= pos.shape[-1] <= MAX_TOPK:
        raise ValueError(f"pos must be [..., k] with k in 1..{MAX_TOPK}, got {tuple(pos.shape)}")
    _check_index(pos, "pos", rows.device)
    lead, k = pos.shape[:-1], pos.shape[-1]
    T = math.prod(lead)
    if rows.dim() != 2 or rows.shape[0] != T * k:
        raise ValueError(f"rows must be [T * k, K] = [{T * k}, K], got {tuple(rows.shape)}")
    if weights is not None:
        if weights.shape != pos.shape:
            raise ValueError(f"weights must be {tuple(pos.shape)}, got {tuple(weights.shape)}")
        if weights.dtype != torch.float32:
            raise TypeError(f"weights must be float32, got {weights.dtype}")
        if weights.device != rows.device:
            raise ValueError("weights must be on the device of rows")
    return lead, T, k, rows.shape[1]


def expert_combine(rows: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] * rows[pos[t, j]] in fp32, rounded once; dropped pairs (negative pos) are left out.

    rows [T * k, K] fp32 or bf16; pos int32 and weights fp32 [..., k] (weights None: ones).  Returns [..., K]; `out`
    may pass a preallocated [T, K]."""
    dt = _dtype_code(rows)
    lead, T, k, K = _combine_sizes(rows, pos, weights)
    if out is not None:
        _check_out(out, "out", (T, K), rows.dtype, rows.device)
    _on_gpu(rows)
    r2, pos = _dense16(rows), pos.contiguous()
    weights = None if weights is None else weights.contiguous()
    y = out if out is not None else torch.empty((T, K), dtype=rows.dtype, device=rows.device)
    _call("swiglu_expert_combine", rows, dt, T, k, K, _p(r2), _p(pos), _p(weights), _p(y))
    return _lead(y, lead, K)


def expert_combine_bwd(dy: torch.Tensor, rows: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor | None = None,
                       out=None):
    """Gradients of expert_combine: (drows [T * k, K], dweights fp32 as weights, None without them).

    drows[pos[t, j]] = weights[t, j] * dy[t] and dweights[t, j] = <dy[t], rows[pos[t, j]]>; zeros for dropped pairs,
    whose rows ~pos names.  pos must be a plan's, which names every row once.  `out` may pass the two preallocated."""
    _same(rows, dy)
    dt = _dtype_code(rows)
    lead, T, k, K = _combine_sizes(rows, pos, weights)
    if tuple(dy.shape) != (*lead, K):
        raise ValueError(f"dy must be {(*lead, K)}, got {tuple(dy.shape)}")
    if out is not None:
        drows, dw = out
        _check_out(drows, "drows", (T * k, K), rows.dtype, rows.device)
        if weights is not None:
            _check_out(dw, "dweights", (T, k), torch.float32, rows.device)
        elif dw is not None:
            raise ValueError("out has an output that this call does not compute")
    _on_gpu(rows)
    r2, d2, pos = _dense16(rows), _dense16(dy), pos.contiguous()
    weights = None if weights is None else weights.contiguous()
    if out is None:
        drows = torch.empty((T * k, K), dtype=rows.dtype, device=rows.device)
        dw = None if weights is None else torch.empty((T, k), dtype=torch.float32, device=rows.device)
    _call("swiglu_expert_combine_bwd", rows, dt, T, k, K, _p(d2), _p(r2), _p(pos), _p(weights), _p(drows), _p(dw))
    return drows, (None if dw is None else _lead(dw, lead, k))


# --------------------------------------------------------- grouped products

def _grouped_weights(w: torch.Tensor, name: str) -> tuple[int, int, int]:
    if w.dim() != 3:
        raise ValueError(f"{name} must be [E, N, K], got {tuple(w.shape)}")
    E, N, K = w.shape
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"{name} must have 1 to {MAX_EXPERTS} experts, got {E}")
    return E, N, K


def _gate_up_sizes(x, wg, wu, offsets, src):
    """(R, E, N, K, T, k) and the checks of grouped_fwd's and grouped_bwd's inputs."""
    _same(x, wg, wu)
    E, N, K = _grouped_weights(wg, "wg")
    if wu.shape != wg.shape:
        raise ValueError(f"wu must have the shape of wg, {tuple(wg.shape)}, got {tuple(wu.shape)}")
    if x.dim() < 1 or x.shape[-1] != K or (src is None and x.dim() != 2):
        raise ValueError(f"x must be [R, {K}] (with src [..., {K}]), got {tuple(x.shape)}")
    T, k = 0, 1
    if src is not None:
        T, k, _ = _tokens_of(x, src)
        R = T * k
    else:
        R = x.shape[0]
    return R, E, N, K, T, k


def _rows_of(x, src, K):
    """x and src as the library takes them: x of 2^31 bytes or more is gathered first."""
    if src is None:
        return _dense16(x), None
    if x.numel() * x.element_size() >= GATHER_BYTES:
        return expert_gather(x, src), None
    return _dense16(x), src.contiguous()


def grouped_fwd(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, offsets: torch.Tensor,
                src: torch.Tensor | None = None, act: str = "silu", out: torch.Tensor | None = None) -> torch.Tensor:
    """The gate/up stage of rows in order of expert, h[r] = act(x_r Wg_e^T) * (x_r Wu_e^T) for the rows
    offsets[e] <= r < offsets[e + 1] of expert e; rows of no expert get zeros.  fp32 or bf16.

    x [R, K] holds the rows, or with src, as expert_plan gives it, the tokens [..., K]: row r is token src[r] // k.
    wg, wu [E, N, K], whose experts may lie apart (w[:, :N] and w[:, N:] of a stacked [E, 2N, K] are taken as they
    are); offsets int32 [E + 1] on the device.  Returns h [R, N]; `out` may pass it preallocated."""
    code = _act_code(act)
    R, E, N, K, T, k = _gate_up_sizes(x, wg, wu, offsets, src)
    dt = _dtype_code(x)
    offsets = _check_offsets(offsets, E, x.device)
    if out is not None:
        _check_out(out, "out", (R, N), x.dtype, x.device)
    _on_gpu(x)
    x2, src = _rows_of(x, src, K)
    wg, sg = _weights16(wg, N, K)
    wu, su = _weights16(wu, N, K)
    h = out if out is not None else torch.empty((R, N), dtype=x.dtype, device=x.device)
    _call("swiglu_grouped_fwd", x, code, dt, R, E, N, K, _p(x2), T, k, _p(src), _p(offsets), _p(wg), sg, _p(wu), su,
          _p(h))
    return h


def grouped_bwd_workspace_bytes(dtype: torch.dtype, R: int, N: int, K: int, gathered: bool = False,
                                E: int | None = None) -> int:
    """Bytes of workspace of grouped_bwd, with src (gathered) or without: for E experts, which often take less, or for
    any number of them."""
    if dtype not in _DT:
        raise TypeError(f"libswiglu supports bfloat16 and float32, got {dtype}")
    if E is None:
        return int(lib().swiglu_grouped_bwd_workspace_bytes(_DT[dtype], R, N, K, int(gathered)))
    return int(lib().swiglu_grouped_bwd_workspace_bytes_of(_DT[dtype], R, E, N, K, int(gathered)))


def grouped_bwd(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, dh: torch.Tensor, offsets: torch.Tensor,
                src: torch.Tensor | None = None, act: str = "silu", workspace: torch.Tensor | None = None, out=None,
                need_dx: bool = True, need_dw: bool = True):
    """Gradients of grouped_fwd: (dx [R, K], dwg, dwu [E, N, K]).

    dx is the rows' also where src is given (the tokens' is expert_combine(dx, pos)); rows of no expert get 0, their
    dh is not read, and experts without rows get 0.  The gradients at the gate's and the up product's outputs are
    rounded to the type of x before dx, dwg and dwu are formed from them.  need_dx or need_dw False leaves those out
    (None).  `out` may pass the three preallocated (None for one that is left out); `workspace` a uint8 device buffer of
    at least grouped_bwd_workspace_bytes(..., E=E) bytes (a smaller or missing one is replaced)."""
    code = _act_code(act)
    R, E, N, K, T, k = _gate_up_sizes(x, wg, wu, offsets, src)
    _same(x, dh)
    dt = _dtype_code(x)
    offsets = _check_offsets(offsets, E, x.device)
    if tuple(dh.shape) != (R, N):
        raise ValueError(f"dh must be {(R, N)}, got {tuple(dh.shape)}")
    if not (need_dx or need_dw):
        raise ValueError("grouped_bwd needs an output")
    if out is not None:
        if len(out) != 3:
            raise ValueError("out must be (dx, dwg, dwu)")
        for t, need, name, shape in zip(out, (need_dx, need_dw, need_dw), ("dx", "dwg", "dwu"),
                                        ((R, K), (E, N, K), (E, N, K))):
            if need:
                _check_out(t, name, shape, x.dtype, x.device)
            elif t is not None:
                raise ValueError("out has an output that this call does not compute")
    _check_workspace(workspace, x.device)
    _on_gpu(x)
    x2, src = _rows_of(x, src, K)
    d2 = _dense16(dh)
    wg, sg = _weights16(wg, N, K)
    wu, su = _weights16(wu, N, K)
    if out is None:
        def new(need, *shape):
            return torch.empty(shape, dtype=x.dtype, device=x.device) if need else None
        out = (new(need_dx, R, K), new(need_dw, E, N, K), new(need_dw, E, N, K))
    dx, dwg, dwu = out
    need = int(lib().swiglu_grouped_bwd_workspace_bytes_of(dt, R, E, N, K, int(src is not None)))
    ws, n = _workspace(workspace, need, x.device)
    _call("swiglu_grouped_bwd", x, code, dt, R, E, N, K, _p(x2), T, k, _p(src), _p(offsets), _p(wg), sg, _p(wu), su,
          _p(d2), _p(dx), _p(dwg), _p(dwu), _p(ws), n)
    return dx, dwg, dwu


def grouped_mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """y[r] = x[r] W_e^T for the rows offsets[e] <= r < offsets[e + 1] of expert e; rows of no expert get zeros.

    x [R, K], w [E, N, K] (experts may lie apart), offsets int32 [E + 1] on the device; fp32 or bf16.  Returns
    [R, N]; `out` may pass it preallocated."""
    _same(x, w)
    dt = _dtype_code(x)
    E, N, K = _grouped_weights(w, "w")
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [R, {K}], got {tuple(x.shape)}")
    R = x.shape[0]
    offsets = _check_offsets(offsets, E, x.device)
    if out is not None:
        _check_out(out, "out", (R, N), x.dtype, x.device)
    _on_gpu(x)
    x2 = _dense16(x)
    w, sw = _weights16(w, N, K)
    y = out if out is not None else torch.empty((R, N), dtype=x.dtype, device=x.device)
    _call("swiglu_grouped_mm", x, dt, R, E, N, K, _p(x2), _p(offsets), _p(w), sw, _p(y))
    return y


def grouped_mm_bwd_workspace_bytes(dtype: torch.dtype, R: int, N: int, K: int, E: int | None = None) -> int:
    """Bytes of workspace of grouped_mm_bwd (0: none is needed), for E experts or for any number of them."""
    if dtype not in _DT:
        raise TypeError(f"libswiglu supports bfloat16 and float32, got {dtype}")
    if E is None:
        return int(lib().swiglu_grouped_mm_bwd_workspace_bytes(_DT[dtype], R, N, K))
    return int(lib().swiglu_grouped_mm_bwd_workspace_bytes_of(_DT[dtype], R, E, N, K))


def grouped_mm_bwd(x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor, out=None,
                   need_dx: bool = True, need_dw: bool = True, workspace: torch.Tensor | None = None):
    """Gradients of grouped_mm: (dx [R, K], dw [E, N, K]); rows of no expert and experts without rows get zeros.
    need_dx or need_dw False leaves one out (None).  `out` may pass the two preallocated, `workspace` a uint8 device
    buffer of at least grouped_mm_bwd_workspace_bytes(..., E=E) bytes (a smaller or missing one is replaced)."""
    _same(x, w, dy)
    dt = _dtype_code(x)
    E, N, K = _grouped_weights(w, "w")
    if x.dim() != 2 or x.shape[1] != K or tuple(dy.shape) != (x.shape[0], N):
        raise ValueError(f"x must be [R, {K}] and dy [R, {N}], got {tuple(x.shape)}, {tuple(dy.shape)}")
    R = x.shape[0]
    offsets = _check_offsets(offsets, E, x.device)
    if not (need_dx or need_dw):
        raise ValueError("grouped_mm_bwd needs an output")
    if out is not None:
        if len(out) != 2:
            raise ValueError("out must be (dx, dw)")
        for t, need, name, shape in zip(out, (need_dx, need_dw), ("dx", "dw"), ((R, K), (E, N, K))):
            if need:
                _check_out(t, name, shape, x.dtype, x.device)
            elif t is not None:
                raise ValueError("out has an output that this call does not compute")
    _check_workspace(workspace, x.device)
    _on_gpu(x)
    x2, d2 = _dense16(x), _dense16(dy)
    w, sw = _weights16(w, N, K)
    if out is None:
        out = (torch.empty((R, K), dtype=x.dtype, device=x.device) if need_dx else None,
               torch.empty((E, N, K), dtype=x.dtype, device=x.device) if need_dw else None)
    dx, dw = out
    ws, n = _workspace(workspace, int(lib().swiglu_grouped_mm_bwd_workspace_bytes_of(dt, R, E, N, K)), x.device)
    _call("swiglu_grouped_mm_bwd", x, dt, R, E, N, K, _p(x2), _p(offsets), _p(w), sw, _p(d2), _p(dx), _p(dw), _p(ws), n)
    return dx, dw


# ----------------------------------------------------------------- autograd

class GroupedSwiGLUFunction(torch.autograd.Function):
    """Autograd wrapper of grouped_fwd on rows (no src).  As in all of these, the gradients have no derivative of
    their own (asking for one raises)."""

    @staticmethod
    def forward(ctx, x, wg, wu, offsets, act="silu"):
        ctx.save_for_backward(x, wg, wu, offsets)
        ctx.act = act
        return grouped_fwd(x, wg, wu, offsets, act=act)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, wg, wu, offsets = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        if not (need_dx or need_dw):
            return (None,) * 5
        dx, dwg, dwu = grouped_bwd(x, wg, wu, dh, offsets, act=ctx.act, need_dx=need_dx, need_dw=need_dw)
        return dx, dwg, dwu, None, None


def grouped_swiglu(x, wg, wu, offsets, act: str = "silu"):
    """Differentiable grouped_fwd of rows [R, K]."""
    return GroupedSwiGLUFunction.apply(x, wg, wu, offsets, act)


class GroupedLinearFunction(torch.autograd.Function):
    """Autograd wrapper of grouped_mm."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return grouped_mm(x, w, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[:2]
        if not (need_dx or need_dw):
            return None, None, None
        dx, dw = grouped_mm_bwd(x, w, dy, offsets, need_dx=need_dx, need_dw=need_dw)
        return dx, dw, None


def grouped_linear(x, w, offsets):
    """Differentiable grouped_mm."""
    return GroupedLinearFunction.apply(x, w, offsets)


class ExpertRowsFunction(torch.autograd.Function):
    """Autograd wrapper of expert_gather; its gradient adds up a token's rows."""

    @staticmethod
    def forward(ctx, x, src, pos):
        ctx.save_for_backward(pos)
        return expert_gather(x, src)

    @staticmethod
    @once_differentiable
    def backward(ctx, drows):
        (pos,) = ctx.saved_tensors
        return expert_combine(drows, pos), None, None


def expert_rows(x, src, pos):
    """Differentiable expert_gather: tokens [..., K] as rows in order of expert, with a plan's src and pos."""
    if tuple(pos.shape[:-1]) != tuple(x.shape[:-1]) or pos.numel() != src.numel():
        raise ValueError(f"pos must be {(*x.shape[:-1], 'k')}, got {tuple(pos.shape)} for src of {src.numel()}")
    return ExpertRowsFunction.apply(x, src, pos)


class ExpertSumFunction(torch.autograd.Function):
    """Autograd wrapper of expert_combine."""

    @staticmethod
    def forward(ctx, rows, pos, weights):
        ctx.save_for_backward(rows, pos, weights)
        return expert_combine(rows, pos, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, pos, weights = ctx.saved_tensors
        drows, dw = expert_combine_bwd(dy, rows, pos, weights)
        return drows, None, dw


def expert_sum(rows, pos, weights=None):
    """Differentiable expert_combine: each token's rows added with the router's weights."""
    return ExpertSumFunction.apply(rows, pos, weights)


class RoutedMLPFunction(torch.autograd.Function):
    """Autograd wrapper of the routed MLP: plan, gate/up with the rows gathered on the way, down, combine."""

    @staticmethod
    def forward(ctx, x, wg, wu, wd, weights, ids, act="silu"):
        E = wg.shape[0]
        offsets, src, pos = expert_plan(ids, E)
        h = grouped_fwd(x, wg, wu, offsets, src=src, act=act)
        rows = grouped_mm(h, wd, offsets)
        ctx.save_for_backward(x, wg, wu, wd, weights, offsets, src, pos, h, rows)
        ctx.act = act
        return expert_combine(rows, pos, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, wg, wu, wd, weights, offsets, src, pos, h, rows = ctx.saved_tensors
        nx, ng, nu, nd, nw = ctx.needs_input_grad[:5]
        out = [None] * 7
        if not any((nx, ng, nu, nd, nw)):
            return tuple(out)
        drows, dw = expert_combine_bwd(dy, rows, pos, weights)
        out[4] = dw if nw else None
        stage = nx or ng or nu
        if stage or nd:
            dh, out[3] = grouped_mm_bwd(h, wd, drows, offsets, need_dx=stage, need_dw=nd)
        if stage:
            dx, out[1], out[2] = grouped_bwd(x, wg, wu, dh, offsets, src=src, act=ctx.act, need_dx=nx,
                                             need_dw=ng or nu)
            if nx:
                out[0] = expert_combine(dx, pos)
        return tuple(out)


def routed_mlp(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, wd: torch.Tensor, ids: torch.Tensor,
               weights: torch.Tensor, act: str = "silu") -> torch.Tensor:
    """The differentiable routed MLP over any number of tokens, fp32 or bf16:

        y[t] = sum_j weights[t, j] * Wd_e (act(Wg_e x[t]) * (Wu_e x[t])),  e = ids[t, j].

    x [..., K]; wg, wu [E, N, K] and wd [E, K, N]; ids int32 and weights fp32 [..., k], as route or router gives them
    (an id outside [0, E) is skipped).  Gradients flow to x, the experts' weights and `weights`.  Between the stages the
    hidden activations, the experts' rows and their gradients are rounded to the type of x.  For a few bf16 tokens
    without gradients moe_fwd is faster, and more exact (16 bits of the hidden activations, fp32 rows)."""
    _same(x, wg, wu, wd)
    _dtype_code(x)
    _act_code(act)
    E, N, K = _grouped_weights(wg, "wg")
    if wu.shape != wg.shape or wd.shape != (E, K, N):
        raise ValueError(f"weights must be [E, N, K], [E, N, K], [E, K, N], got {tuple(wg.shape)}, "
                         f"{tuple(wu.shape)}, {tuple(wd.shape)}")
    if x.dim() < 1 or x.shape[-1] != K:
        raise ValueError(f"x must be [..., {K}], got {tuple(x.shape)}")
    if ids.dim() < 1 or ids.shape[:-1] != x.shape[:-1] or ids.shape != weights.shape:
        raise ValueError(f"ids and weights must be {(*x.shape[:-1], 'k')}, got {tuple(ids.shape)}, "
                         f"{tuple(weights.shape)}")
    _check_index(ids, "ids", x.device)
    if weights.dtype != torch.float32 or weights.device != x.device:
        raise TypeError(f"weights must be float32 on {x.device}, got {weights.dtype} on {weights.device}")
    _on_gpu(x)
    return RoutedMLPFunction.apply(x, wg, wu, wd, weights, ids, act)


# ------------------------------------------------------ gradients' norm, clip

def _packed(t: torch.Tensor) -> bool:
    """Whether t's elements fill its span of memory, each place once, in some order of the dimensions."""
    at = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != at:
            return False
        at *= size
    return True


def _apart(t: torch.Tensor) -> bool:
    """Whether no two elements of t share a place: every stride passes what the smaller ones reach."""
    reach = 0
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride <= reach:
            return False
        reach += stride * (size - 1)
    return True


def _dims(t: torch.Tensor) -> list:
    """(stride in bytes, steps) of t's dimensions, the longest stride first."""
    size = t.element_size()
    return sorted(((s * size, n - 1) for s, n in zip(t.stride(), t.shape) if s != 0 and n != 1), reverse=True)


def _span(t: torch.Tensor) -> tuple[int, int]:
    """t's first byte and the end of its last."""
    at, size = t.data_ptr(), t.element_size()
    return at, at + size * (t.numel() if t.is_contiguous() else sum(s * (n - 1) for s, n in zip(t.stride(), t.shape)) + 1)


def _crossing(tensors: list):
    """Pairs (i, j) of tensors that may share memory: their spans cross.  Among views whose outermost strides are equal
    and whose parts below them do not wrap round that stride (slices of one tensor), these parts' spans cross."""
    def sweep(spans):
        order = sorted(spans, key=spans.get)
        for at, i in enumerate(order):
            for j in itertools.islice(order, at + 1, None):
                if spans[j][0] >= spans[i][1]:
                    break
                yield i, j

    def pairs(group):
        outer = {i: (_dims(tensors[i]) or [(0, 0)])[0] for i in group}
        period, base = outer[group[0]][0], spans[group[0]][0]
        if period and all(s == period for s, _ in outer.values()):
            parts = {}
            for i, (_, n) in outer.items():
                low = (spans[i][0] - base) % period
                parts[i] = (low, low + spans[i][1] - spans[i][0] - period * n)
            if max(end for _, end in parts.values()) <= period:
                return sweep(parts)
        return sweep({i: spans[i] for i in group})

    spans = list(map(_span, tensors))
    group, end = [], 0
    for i in sorted(range(len(tensors)), key=spans.__getitem__):
        if spans[i][0] >= end:
            if len(group) > 1:
                yield from pairs(group)
            group = []
        group.append(i)
        end = max(end, spans[i][1])
    if len(group) > 1:
        yield from pairs(group)


def _share(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors have a byte in common: whether, over both, strides times indices (b's counted from its end)
    and bytes inside an element add up to the distance from a's first byte to b's last.  (True also where that is not
    told in 20000 steps.)"""
    first, sizes = a.data_ptr(), (a.element_size(), b.element_size())
    unit = math.gcd(*sizes, first - b.data_ptr())
    count = {1: sum(sizes) // unit - 2}
    for s, n in _dims(a) + _dims(b):
        count[s // unit] = count.get(s // unit, 0) + n
    terms = sorted(count.items(), reverse=True)
    reach = [sum(s * n for s, n in terms[i:]) for i in range(len(terms) + 1)]
    common = [math.gcd(*(s for s, n in terms[i:] if n)) for i in range(len(terms) + 1)]
    steps = 20000

    def adds_up(i, to):
        nonlocal steps
        steps -= 1
        if steps < 0:
            return True
        if not 0 <= to <= reach[i]:
            return False
        if to in (0, reach[i]):
            return True
        if to % common[i]:                       # (0 < to < reach[i]: some term is left)
            return False
        s, n = terms[i]
        return any(adds_up(i + 1, to - s * x) for x in range(max(0, -((reach[i + 1] - to) // s)), min(n, to // s) + 1))
    return adds_up(0, (_span(b)[1] - first) // unit - 1)


def _overlap(written: list, read: list | None = None):
    """Two of the tensors that share memory, as (list, index) pairs, list 0 for written and 1 for read, or None.  What
    is written may be what is read at the same index, element by element."""
    at = [(side, i) for side, ts in enumerate((written, read or [])) for i, t in enumerate(ts) if t.numel()]
    tensors = [(written, read)[side][i] for side, i in at]
    for a, b in _crossing(tensors):
        (side, i), (other, j) = at[a], at[b]
        if side == other == 1:
            continue
        if side != other and i == j and _same_place(tensors[a], tensors[b]):
            continue
        if _share(tensors[a], tensors[b]):
            return min(at[a], at[b]), max(at[a], at[b])
    return None


def _same_place(a: torch.Tensor, b: torch.Tensor) -> bool:
    return a.data_ptr() == b.data_ptr() and all(n == 1 or s == t for n, s, t in zip(a.shape, a.stride(), b.stride()))


def _grad_list(grads) -> list:
    return [grads] if isinstance(grads, torch.Tensor) else list(grads)


def _grad_codes(grads: list) -> tuple[array, torch.device]:
    """The dtype codes of gradients on one device, and that device.  (Each pass over a list of hundreds of tensors
    takes longer on the host than the kernels on the GPU, so there is one for each question.)"""
    if not grads:
        raise ValueError("no gradients were given")
    kinds = list(map(attrgetter("dtype"), grads))
    if kinds.count(kinds[0]) == len(kinds):
        codes = array("i", [_dtype_code(grads[0])]) * len(kinds)
    else:
        codes = array("i", map(_dtype_code, grads))
    where = set(map(torch.Tensor.get_device, grads))
    if len(where) > 1:
        raise ValueError(f"gradients must be on one device, got {sorted({str(g.device) for g in grads})}")
    return codes, grads[0].device


def _grad_arrays(grads: list) -> tuple[array, array]:
    """Addresses and sizes; host arrays that must live until the call returns."""
    return array("Q", map(torch.Tensor.data_ptr, grads)), array("q", map(torch.Tensor.numel, grads))


def _addr(a) -> int | None:
    return None if a is None else a.buffer_info()[0]


def grad_norm_workspace_bytes(count: int) -> int:
    """Bytes of workspace of grad_norm and clip_grads for `count` tensors."""
    return int(lib().swiglu_grad_norm_workspace_bytes(count))


def grad_norm(grads, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The 2-norm of all elements of the tensors `grads` together (fp32 and bf16 mixed), a 0-dim fp32 tensor.  Squares
    are formed and added in fp64."""
    grads = _grad_list(grads)
    codes, dev = _grad_codes(grads)
    _check_workspace(workspace, dev)
    _on_gpu(grads[0])
    if not all(map(torch.Tensor.is_contiguous, grads)):
        grads = [t if t.is_contiguous() or _packed(t) else t.contiguous() for t in grads]
    at, n = _grad_arrays(grads)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws, size = _workspace(workspace, int(lib().swiglu_grad_norm_workspace_bytes(len(grads))), dev)
    _call("swiglu_grad_norm", norm, len(grads), _addr(codes), _addr(at), _addr(n), _p(norm), _p(ws), size)
    return norm


@torch.no_grad()
def clip_grads(grads, max_norm: float, eps: float = 1e-6, out=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Scales the tensors `grads` together to a 2-norm of at most max_norm, g *= min(1, max_norm / (norm + eps)), and
    returns the norm they had (0-dim fp32), without waiting for the GPU.

    In place, or into the tensors `out` of the same shapes and types (out[i] may be grads[i]).  fp32 and bf16 may be
    mixed; tensors that overlap each other or are given twice are refused.  A norm that is NaN makes every gradient
    NaN; an infinite one makes finite elements 0 and infinite ones NaN.  An infinite max_norm clips nothing (but NaN
    norms), and a norm + eps of 0 leaves the zeros.  `workspace` may pass a uint8 device buffer of at least
    grad_norm_workspace_bytes(len(grads)) bytes (a smaller or missing one is replaced)."""
    grads = _grad_list(grads)
    codes, dev = _grad_codes(grads)
    max_norm, eps = float(max_norm), float(eps)
    to = None
    if out is not None:
        to = _grad_list(out)
        if len(to) != len(grads):
            raise ValueError(f"out must have {len(grads)} tensors, got {len(to)}")
        for i, (t, g) in enumerate(zip(to, grads)):
            if t.shape != g.shape or t.dtype != g.dtype or t.device != dev:
                raise ValueError(f"out[{i}] must be {tuple(g.shape)}, {g.dtype} on {dev}, got {tuple(t.shape)}, {t.dtype} "
                                 f"on {t.device}")
    written = to if to is not None else grads
    _check_workspace(workspace, dev)
    back = []                                    # (tensor, its contiguous stand-in): copied back after the call
    if not (all(map(torch.Tensor.is_contiguous, grads)) and (to is None or all(map(torch.Tensor.is_contiguous, to)))):
        for i, t in enumerate(written):
            if not (t.is_contiguous() or _apart(t)):
                raise ValueError(f"{'out' if to is not None else 'grads'}[{i}] has elements that share memory, strides {t.stride()}")
        # Here, since the library sees the stand-ins (contiguous tensors it checks itself).
        both = _overlap(written, grads if to is not None else None)
        if both is not None:
            a, b = (f"{'grads' if to is None or side else 'out'}[{i}]" for side, i in both)
            raise ValueError(f"{a} and {b} overlap")
        src, dst = list(grads), list(written)
        for i, (g, t) in enumerate(zip(grads, written)):
            if (g.is_contiguous() and t.is_contiguous()) or (g.stride() == t.stride() and _packed(g)):
                continue
            src[i] = g.contiguous()
            dst[i] = src[i] if to is None else t if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=dev)
            if dst[i] is not t:
                back.append((t, dst[i]))
        grads, written = src, dst
    _on_gpu(grads[0])
    at, n = _grad_arrays(grads)
    dst = None if to is None else array("Q", map(torch.Tensor.data_ptr, written))
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws, size = _workspace(workspace, int(lib().swiglu_grad_norm_workspace_bytes(len(grads))), dev)
    _call("swiglu_clip_grads", norm, len(grads), _addr(codes), _addr(at), _addr(n), _addr(dst), max_norm, eps, _p(norm),
          _p(ws), size)
    for t, c in back:
        if t.is_inference():                     # written in that mode only
            with torch.inference_mode():
                t.copy_(c)
        else:
            t.copy_(c)
    try:
        torch.autograd.graph.increment_version(written)
    except RuntimeError:                         # tensors made in inference mode count no versions
        torch.autograd.graph.increment_version([t for t in written if not t.is_inference()])
    return norm
