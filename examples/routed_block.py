"""A routed SwiGLU block from the library's entry points: trained, then served token by token.

    python examples/routed_block.py

train() fits one block to a synthetic target: the norms around it (block_norms), the router (router) and, expert by
expert, the fused gate/up stage (swiglu), all with their HIP backward passes.  decode() runs a stack of blocks on a
few tokens a step: route, moe_fwd, and one block_norm between blocks that joins the block's output to the residual
stream and forms the next block's input.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import swiglu_mlp_fwd_amd as S  # noqa: E402

DEV = "cuda"


def train(steps=40, tokens=512, width=256, hidden=384, experts=8, topk=2, lr=3e-3, seed=0):
    """Returns the first and the last loss."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def param(*shape, std=0.05, mean=0.0):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).requires_grad_(True)
    w_in, w_out, gate = param(width, mean=1.0), param(width, mean=1.0), param(width, mean=1.0)
    wr = param(width, experts)
    wg = [param(hidden, width) for _ in range(experts)]
    wu = [param(hidden, width) for _ in range(experts)]
    wd = [param(width, hidden) for _ in range(experts)]
    opt = torch.optim.Adam([w_in, w_out, gate, wr, *wg, *wu, *wd], lr=lr)
    x = torch.randn((tokens, width), generator=g, device=DEV)
    target = x + torch.sin(x @ (torch.randn((width, width), generator=g, device=DEV) / width ** 0.5))
    losses = []
    for _ in range(steps):
        _, z = S.block_norms(x, w_in=w_in)
        w, ids = S.router(z @ wr, topk)
        y = torch.zeros_like(x)
        for e in range(experts):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            h = S.swiglu(z[t], wg[e], wu[e])
            y = y.index_add(0, t, w[t, j].unsqueeze(1) * (h @ wd[e].t()))
        out, _ = S.block_norms(x, y, w_out, gate)
        loss = (out - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses[0], losses[-1]


def decode(steps=8, batch=8, blocks=4, width=1024, hidden=512, experts=16, topk=4, seed=1):
    """`steps` passes of `batch` tokens through a stack of routed blocks; returns the last step's outputs."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def weight(*shape, std=0.03):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)
    ones = torch.ones(width, device=DEV, dtype=torch.bfloat16)
    layers = [dict(wr=weight(width, experts).float(), wg=weight(experts, hidden, width),
                   wu=weight(experts, hidden, width), wd=weight(experts, width, hidden)) for _ in range(blocks)]
    ws = torch.empty(S.moe_workspace_bytes(batch, hidden, width, topk), dtype=torch.uint8, device=DEV)
    x = weight(batch, width, std=1.0)
    for _ in range(steps):
        res, (_, z) = x, S.block_norm(x, w_in=ones)
        for p in layers:
            w, ids = S.route(z.float() @ p["wr"], topk)
            y = S.moe_fwd(z, p["wg"], p["wu"], p["wd"], ids, w, workspace=ws)
            res, z = S.block_norm(res, y, w_out=ones, w_in=ones, scale=blocks ** -0.5)
        x = z
    return x


if __name__ == "__main__":
    first, last = train()
    print(f"train: loss {first:.4f} -> {last:.4f}")
    y = decode()
    torch.cuda.synchronize()
    print(f"decode: {tuple(y.shape)}, rms {y.float().square().mean().sqrt().item():.3f}")
