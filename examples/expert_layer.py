"""An expert layer trained and served with the library's operators, and a
shared projection with a low-rank adapter per request.

    logits = x Wr^T;  (p, ids) = the k largest, softmax over them
    y[t] = sum_j p[t, j] * expert_ids[t, j](x[t]),
    expert_e(x) = (silu(x Wg_e^T) * (x Wu_e^T)) Wd_e^T

Forward: route_topk chooses, expert_sort gives every (token, choice) pair its
row, expert_dispatch_quant brings the tokens there as E4M3, grouped_gemm_contiguous
forms gate and up (one product) and the down projection, expert_combine brings
the rows back.  Backward: expert_combine_grad, per expert gated_nt_grad and two
plain torch products, expert_combine of the rows' gradients (the dispatch's
gradient), route_topk_grad; clip_grad_norm clips all gradients.

Serving a step of single tokens takes the masked layout, whose shapes do not
depend on the choice, so that it can be captured in a graph.  Behind it a
shared output projection (gemm_nt) serves requests that each have their own
adapter (adapter_rows, add_adapters).

    python examples/expert_layer.py [--tokens 512] [--width 512] [--hidden 512] [--experts 8] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_block_e4m3_amd as fp8  # noqa: E402


def plain_layer(x, wr, wg, wu, wd, k):
    """The layer in plain torch, expert by expert (FP32 or FP64; differentiable)."""
    p, ids = (x @ wr.t()).topk(k, dim=1)
    p = torch.softmax(p, 1)
    y = torch.zeros_like(x)
    for e in range(wg.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g = x[t] @ wg[e].t()
        y = y.index_add(0, t, p[t, j, None] * ((g * torch.sigmoid(g) * (x[t] @ wu[e].t())) @ wd[e].t()))
    return y


def quantized(w):
    """E4M3 codes and scales of weights (E, N, K)."""
    E, N, K = w.shape
    q, s = fp8.quant_128x128(w.reshape(E * N, K))
    return q.view(E, N, K), s.view(E, N // 128, K // 128)


def experts(xq, sa, gate_up, down, product):
    """Both of the experts' products; returns (y, the projections' BF16 rows, h)."""
    gu = product(xq, sa, *gate_up)
    g, u = gu.float().chunk(2, dim=-1)
    h = g * torch.sigmoid(g) * u
    hq, sh = fp8.quant_1x128(h.reshape(-1, h.shape[-1]))
    return product(hq.view(h.shape), sh, *down), gu, h


def forward(x, wr, gate_up, down, k):
    """The layer for a batch of tokens; returns y and what the gradient needs."""
    E = down[0].shape[0]
    logits = x @ wr.t()
    p, ids = fp8.route_topk(logits, k)
    pos, src, m_indices, counts = fp8.expert_sort(ids, E)
    xq, sa = fp8.expert_dispatch_quant(x, pos, src.shape[0])
    rows, gu, h = experts(xq, sa, gate_up, down, lambda a, s, w, sb: fp8.grouped_gemm_contiguous(a, s, w, sb, m_indices))
    return fp8.expert_combine(rows, pos, p), (logits, p, ids, pos, src, counts, rows, gu, h)


def gradients(x, dy, wr, wg, wu, wd, saved):
    """(dx, dwr, dwg, dwu, dwd) of a loss whose gradient at y is dy."""
    logits, p, ids, pos, src, counts, rows, gu, h = saved
    drows, dp = fp8.expert_combine_grad(dy.bfloat16(), rows, pos, p, src)
    dlogits = fp8.route_topk_grad(dp, logits, ids)
    xs = fp8.expert_dispatch(x.bfloat16(), pos, src)
    dxs = torch.zeros_like(xs)
    dwg, dwu, dwd = (torch.zeros_like(w) for w in (wg, wu, wd))
    F = wg.shape[1]
    at = 0
    for e, n in enumerate(counts.tolist()):
        r = slice(at, at + n)
        at += (n + 127) // 128 * 128
        if n == 0:
            continue
        d = drows[r].float()
        dwd[e] = d.t() @ h[r]
        dh = (d @ wd[e]).bfloat16()
        dxs[r], a, b = fp8.gated_nt_grad(dh, gu[r, :F].contiguous(), gu[r, F:].contiguous(), xs[r], wg[e].bfloat16(), wu[e].bfloat16())
        dwg[e], dwu[e] = a, b
    dx = fp8.expert_combine(dxs, pos).float() + dlogits @ wr
    return dx, dlogits.t() @ x, dwg, dwu, dwd


def serve_tokens(x, wr, gate_up, down, k, max_m):
    """The layer for a step of single tokens, in the masked layout."""
    E = down[0].shape[0]
    p, ids = fp8.route_topk(x @ wr.t(), k)
    pos, _, masked_m = fp8.expert_sort_masked(ids, E, max_m)
    xq, sa = fp8.expert_dispatch_quant(x, pos, (E, max_m))
    rows, _, _ = experts(xq, sa, gate_up, down, lambda a, s, w, sb: fp8.grouped_gemm_masked(a, s, w, sb, masked_m))
    return fp8.expert_combine(rows, pos, p)


def project(x, weight, adapters, requests):
    """A shared projection of BF16 tokens, each with its request's adapter added."""
    xq, sa = fp8.quant_1x128(x.float())
    y = fp8.gemm_nt(xq, sa, *weight)
    a, b, scale = adapters
    return fp8.add_adapters(x, a, b, scale, fp8.adapter_rows(requests, a.shape[0]), y, out=y)


def main(tokens: int = 512, width: int = 512, hidden: int = 512, experts: int = 8, steps: int = 20, log=print) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, std):
        return torch.randn(shape, generator=gen, device="cuda") * std

    def new_weights():
        return [rand(experts, width, std=width ** -0.5), rand(experts, hidden, width, std=width ** -0.5),
                rand(experts, hidden, width, std=width ** -0.5), rand(experts, width, hidden, std=hidden ** -0.5)]

    k = min(2, experts)
    teacher, weights = new_weights(), new_weights()
    x = rand(tokens, width, std=1.0)
    target = plain_layer(x, *teacher, k)
    losses = []
    for step in range(steps):
        wr, wg, wu, wd = weights
        y, saved = forward(x, wr, quantized(torch.cat((wg, wu), 1)), quantized(wd), k)
        err = y.float() - target
        grads = list(gradients(x, err * (2.0 / err.numel()), wr, wg, wu, wd, saved)[1:])
        norm = fp8.clip_grad_norm(grads, 0.02)
        for w, d in zip(weights, grads):
            w -= 20.0 * d
        losses.append(float((err * err).mean()))
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}")

    wr, wg, wu, wd = weights
    gate_up, down = quantized(torch.cat((wg, wu), 1)), quantized(wd)
    ref = plain_layer(x[:16], *weights, k)
    served = serve_tokens(x[:16], wr, gate_up, down, k, 128)
    error = float((served.float() - ref).square().mean().sqrt() / ref.square().mean().sqrt())
    log(f"served 16 tokens: error {error:.3f} of the layer's own root mean square")

    R = 16
    adapters = (rand(4, R, width, std=width ** -0.5).bfloat16(), rand(4, width, R, std=0.2).bfloat16(),
                torch.ones(4, device="cuda"))
    requests = torch.tensor([0, 1, 2, 3, 0, -1, 2, 2, 1, 1, 1, 0, 3, -1, 3, 0], dtype=torch.int32, device="cuda")
    out = project(served, fp8.quant_128x128(rand(width, width, std=width ** -0.5)), adapters, requests)
    log(f"projected with {adapters[0].shape[0]} adapters: {tuple(out.shape)}")
    return {"losses": losses, "error": error, "out": out}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("width", 512), ("hidden", 512), ("experts", 8), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    main(**vars(ap.parse_args()))
