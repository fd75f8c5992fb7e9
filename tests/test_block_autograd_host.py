"""The autograd forms of the router and the norms without a GPU, over stand-ins for the library's calls."""
import pytest
import torch

import swiglu_mlp_fwd_amd.block_ops as ops


@torch.no_grad()
def softmax_choice(logits, k, score="softmax", renorm=True, scale=1.0, out=None):
    w, ids = torch.softmax(logits, -1).topk(k)
    return w, ids.to(torch.int32)


@torch.no_grad()
def softmax_grad(logits, ids, dw, score="softmax", renorm=True, scale=1.0, out=None):
    p = torch.softmax(logits, -1)
    d = torch.zeros_like(p).scatter_add(1, ids.long(), dw)
    return p * (d - (p * d).sum(-1, keepdim=True))


def test_router_refuses_a_second_derivative(monkeypatch):
    """The gradients have no derivative of their own; where one is asked for, that is an error and not a zero."""
    monkeypatch.setattr(ops, "route", softmax_choice)
    monkeypatch.setattr(ops, "route_bwd", softmax_grad)
    l = torch.randn(4, 8, requires_grad=True)
    w, _ = ops.router(l, 2)
    (d,) = torch.autograd.grad(w.square().sum(), l, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (w.sum() + d.square().sum()).backward()
    w, _ = ops.router(l, 2)                      # the first derivative is as ever
    w[:, 0].sum().backward()
    _, ids = softmax_choice(l.detach(), 2)
    assert torch.equal(l.grad, softmax_grad(l.detach(), ids, torch.tensor([[1.0, 0.0]]).expand(4, 2)))


@torch.no_grad()
def scaled(res, y=None, w_in=None, **kw):
    return None, res * w_in


@torch.no_grad()
def scaled_grad(ro, y=None, w_in=None, dz=None, **kw):
    return dz * w_in, None, None, None, (dz * ro).sum(0)


def test_block_norms_refuse_a_second_derivative(monkeypatch):
    monkeypatch.setattr(ops, "block_norm", scaled)
    monkeypatch.setattr(ops, "block_norm_bwd", scaled_grad)
    x, w = torch.randn(3, 5, requires_grad=True), torch.randn(5, requires_grad=True)
    _, z = ops.block_norms(x, w_in=w)
    (dx,) = torch.autograd.grad(z.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (z.sum() + dx.square().sum()).backward()
    _, z = ops.block_norms(x, w_in=w)
    z.sum().backward()
    assert torch.equal(x.grad, w.detach().expand(3, 5)) and torch.equal(w.grad, x.detach().sum(0))
