"""A mixture-of-experts feed-forward layer in MXFP4: trained, then decoded.

Each token goes to its `topk` experts; expert e computes W2_e silu(W1_e x).
Both projections are MXFP4 products by expert whose operands are cast from bf16
on the way, forward and backward, with fp32 master weights; the routing stays
on the device (no counts come to the host).  After training, the layer keeps
MXFP4 weights alone and decodes single tokens.

    python examples/mxfp4_experts.py [--tokens 4096 --hidden 1024 --inner 2048 --experts 16 --topk 2 --steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_bf16_amd as nv  # noqa: E402


def cast_weights(w, rowwise=True, columnwise=True):
    """MXFP4 operands of stacked weights [E, N, K] as the grouped products take
    them: rows (sums over K) and columns (sums over N)."""
    outs = [nv.mx_quantize(e, rowwise, columnwise) for e in w.to(torch.bfloat16)]
    return {k: torch.stack([o[k] for o in outs]) for k in outs[0]}


class ExpertLinear(torch.autograd.Function):
    """y[r] = x[rows[r]] W_e^T for the rows r of expert e (every row of x
    without `rows`)."""

    @staticmethod
    def forward(ctx, x, w, offsets, rows):
        q = cast_weights(w)
        ctx.save_for_backward(x, q["col_q"], q["col_sf"], offsets, rows)
        return nv.mx_linear_grouped(x, q["row_q"], q["row_sf"], offsets, rows=rows)

    @staticmethod
    def backward(ctx, dy):
        x, wt_q, wt_sf, offsets, rows = ctx.saved_tensors
        d = nv.mx_quantize_grouped(dy.contiguous(), offsets)
        q = nv.mx_quantize_grouped(x, offsets, rows=rows, rowwise=False)
        dw = nv.mx_wgrad_grouped(d["col_q"], d["col_sf"], q["col_q"], q["col_sf"], offsets)
        dx = nv.mx_gemm_grouped(d["row_q"], d["row_sf"], wt_q, wt_sf, offsets)
        if rows is not None:          # a token's rows add up
            dx = torch.zeros(x.shape, dtype=torch.float32, device=x.device).index_add_(0, rows, dx.float()).to(x.dtype)
        return dx, dw, None, None


def route(x, router, topk):
    """Rows sorted by expert: offsets [E + 1] and rows [T topk] (int32, on the
    device), each row's weight, and its place in the sorted order."""
    p, ids = torch.softmax(x.float() @ router.t(), 1).topk(topk, 1)
    order = torch.argsort(ids.reshape(-1), stable=True)
    counts = torch.zeros(router.shape[0], dtype=torch.int32, device=x.device)
    counts.scatter_add_(0, ids.reshape(-1), torch.ones_like(ids.reshape(-1), dtype=torch.int32))
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
    return offsets, (order // topk).int(), (p / p.sum(1, keepdim=True)).reshape(-1)[order], order


def layer(x, router, w1, w2, topk):
    offsets, rows, p, _ = route(x, router, topk)
    h = torch.nn.functional.silu(ExpertLinear.apply(x, w1, offsets, rows))
    y = ExpertLinear.apply(h, w2, offsets, None)
    return torch.zeros(x.shape[0], w2.shape[1], device=x.device).index_add(0, rows, y.float() * p[:, None])


def decode(x, router, q1, q2, topk):
    """The layer on a few tokens, from MXFP4 weights; the rows' weights go into
    the second product."""
    offsets, rows, p, order = route(x, router, topk)
    h = torch.nn.functional.silu(nv.mx_linear_grouped(x, q1["row_q"], q1["row_sf"], offsets, rows=rows))
    y = nv.mx_linear_grouped(h, q2["row_q"], q2["row_sf"], offsets, row_scale=p, out_dtype=torch.float32)
    back = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=x.device))
    return y[back].view(x.shape[0], topk, -1).sum(1)


def train(tokens=4096, hidden=1024, inner=2048, experts=16, topk=2, steps=20, seed=0, lr=0.05, log=print):
    """Fits random targets; returns the losses and the trained parameters."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    router = rand(experts, hidden) * hidden ** -0.5
    w1 = (rand(experts, inner, hidden) * hidden ** -0.5).requires_grad_()
    w2 = (rand(experts, hidden, inner) * inner ** -0.5).requires_grad_()
    x = rand(tokens, hidden).bfloat16()
    target = torch.tanh(x.float() @ rand(hidden, hidden) * hidden ** -0.5)
    opt = torch.optim.SGD([w1, w2], lr=lr * tokens, momentum=0.9)
    losses = []
    for step in range(steps):
        loss = (layer(x, router, w1, w2, topk) - target).square().mean(1).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        log(f"step {step}: loss {losses[-1]:.4f}")
    return losses, router, w1.detach(), w2.detach(), x


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 1024), ("inner", 2048), ("experts", 16), ("topk", 2), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    _, router, w1, w2, x = train(a.tokens, a.hidden, a.inner, a.experts, a.topk, a.steps)
    q1, q2 = cast_weights(w1, columnwise=False), cast_weights(w2, columnwise=False)
    size = sum(t.numel() for q in (q1, q2) for t in q.values())
    y = decode(x[:1], router, q1, q2, a.topk)
    whole = layer(x, router, w1, w2, a.topk)[:1]
    print(f"MXFP4 weights: {size / 1e6:.1f} MB; one token decoded, "
          f"{float((y - whole).norm() / whole.norm()):.1e} from the trained layer's output")


if __name__ == "__main__":
    main()
