"""A gated feed-forward layer y = (act(x Wg^T) * (x Wu^T)) Wd^T, trained and
then served with the library's operators.

Training step: the weights and activations are quantized to block-scaled E4M3,
gated_nt forms h and keeps the projections, gemm_nt is the down projection;
backward, gated_nt_grad takes the gradient through the gated block in BF16 (the
down projection's own gradient is two plain torch products) and clip_grad_norm
clips all gradients in place before the update of the FP32 weights.

Serving: a prompt goes through gated_nt_qout, whose quantized output is the
down projection's operand; then single tokens through 4-bit weights,
gated_gemv_w4 and gemv_w4.

    python examples/gated_ffn.py [--tokens 512] [--width 512] [--hidden 1024] [--steps 30]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_block_e4m3_amd as fp8  # noqa: E402


def layer(x, wg, wu, wd):
    """The layer in plain FP32."""
    g = x @ wg.t()
    return (g * torch.sigmoid(g) * (x @ wu.t())) @ wd.t()


def train_step(x, target, weights, lr, max_norm):
    """One step on (x, target); returns the loss and the gradient norm."""
    wg, wu, wd = weights
    xq, sa = fp8.quant_1x128(x)
    wgq, sg = fp8.quant_128x128(wg)
    wuq, su = fp8.quant_128x128(wu)
    wdq, sd = fp8.quant_128x128(wd)
    h, g, u = fp8.gated_nt(xq, sa, wgq, sg, wuq, su, save=True)
    hq, sh = fp8.quant_1x128(h.float())
    y = fp8.gemm_nt(hq, sh, wdq, sd).float()
    err = y - target
    dy = err * (2.0 / err.numel())
    dh = (dy @ wd).bfloat16()
    dwd = dy.t() @ h.float()
    _, dwg, dwu = fp8.gated_nt_grad(dh, g, u, x.bfloat16(), wg.bfloat16(), wu.bfloat16(), need_dx=False)
    grads = [dwg, dwu, dwd]
    norm = fp8.clip_grad_norm(grads, max_norm)
    for w, d in zip(weights, grads):
        w -= lr * d.float()
    return float((err * err).mean()), float(norm)


def serve_prompt(x, wg, wu, wd):
    """A prompt through E4M3 weights: h leaves the gated block quantized."""
    xq, sa = fp8.quant_1x128(x)
    hq, sh = fp8.gated_nt_qout(xq, sa, *fp8.quant_128x128(wg), *fp8.quant_128x128(wu))
    return fp8.gemm_nt(hq, sh, *fp8.quant_128x128(wd))


def four_bit(w, fmt):
    """(codes, scales, zero points) of a weight."""
    return fp8.quant_int4(w, group=64) if fmt == "int4" else (*fp8.quant_mxfp4(w), None)


def serve_tokens(x, gate, up, down):
    """Up to 16 tokens through 4-bit weights."""
    h = fp8.gated_gemv_w4(x, gate[0], gate[1], up[0], up[1], zeros_g=gate[2], zeros_u=up[2])
    return fp8.gemv_w4(h, down[0], down[1], zeros=down[2])


def main(tokens: int = 512, width: int = 512, hidden: int = 1024, steps: int = 30, log=print) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(0)

    def rand(r, c, s):
        return torch.randn((r, c), generator=gen, device="cuda") * s

    def new_weights():
        return [rand(hidden, width, width ** -0.5), rand(hidden, width, width ** -0.5), rand(width, hidden, hidden ** -0.5)]

    teacher, weights = new_weights(), new_weights()
    x = rand(tokens, width, 1.0)
    target = layer(x, *teacher)
    losses = []
    for step in range(steps):
        loss, norm = train_step(x, target, weights, lr=20.0, max_norm=0.02)
        losses.append(loss)
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}  loss {loss:.4f}  gradient norm {norm:.4f}")

    ref = layer(x, *weights)
    scale = float(ref.square().mean().sqrt())
    errors = {"prompt": float((serve_prompt(x, *weights).float() - ref).square().mean().sqrt()) / scale}
    for fmt in ("int4", "mxfp4"):
        packed = [four_bit(w, fmt) for w in weights]
        y = torch.cat([serve_tokens(x[i:i + 1].bfloat16(), *packed) for i in range(4)])
        errors[fmt] = float((y.float() - ref[:4]).square().mean().sqrt()) / scale
    for name, e in errors.items():
        log(f"served ({name}): error {e:.3f} of the layer's own root mean square")
    return {"losses": losses, "errors": errors}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("width", 512), ("hidden", 1024), ("steps", 30)):
        ap.add_argument("--" + name, type=int, default=default)
    main(**vars(ap.parse_args()))
