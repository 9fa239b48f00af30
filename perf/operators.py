"""Benchmark cases of the feed-forward operators: the gated feed-forward block
(forward on block-scaled E4M3 operands, backward in BF16), matrix-vector
products with 4-bit weights and group scales, and the global gradient norm
with clipping.

Each case runs in a plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through the library's entry points; ``exact`` computes the
same outputs in 64 bits from the definitions.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

LARGEST_FLOPS = 4 * 8192 * 4096 * 7168      # the largest listed product
LARGEST_ELEMENTS = 400 << 20                # the largest listed set of gradients


def listed():
    """The listed cases.  K = 7168 with N = 2048 is the gate / up projection
    of the 8-expert workload (its 4096 columns are both), K = 2048 with
    N = 7168 the matching down projection, 24576 the widest decode product and
    2112 the narrowest."""
    return [
        # one token through the gate and up projections while serving: latency
        {"name": "gated token", "op": "gated", "M": 1, "N": 2048, "K": 7168, "act": "silu", "out": "bf16", "pow2": False},
        # a small ragged batch of tokens, an N that is no multiple of 128
        {"name": "gated decode ragged", "op": "gated", "M": 37, "N": 2112, "K": 1536, "act": "gelu", "out": "bf16", "pow2": False},
        # a training micro-batch: h and the saved g and u
        {"name": "gated train", "op": "gated", "M": 4096, "N": 2048, "K": 7168, "act": "silu", "out": "save", "pow2": False},
        # a long prefill whose output is quantized for the down projection
        {"name": "gated prefill quantized", "op": "gated", "M": 8192, "N": 4096, "K": 7168, "act": "silu", "out": "quant", "pow2": True},
        # gradients of a small odd-sized block
        {"name": "grad odd", "op": "grad", "M": 777, "N": 500, "K": 640, "act": "gelu"},
        # gradients of a short ragged sequence against wide weights
        {"name": "grad short", "op": "grad", "M": 500, "N": 2112, "K": 7168, "act": "silu"},
        # gradients of the training micro-batch above
        {"name": "grad train", "op": "grad", "M": 4096, "N": 2048, "K": 7168, "act": "silu"},
        # one token through the down projection of one expert, MXFP4 weights: latency
        {"name": "gemv token", "op": "gemv", "M": 1, "N": 7168, "K": 2048, "fmt": "mxfp4", "group": 32, "zeros": False, "gated": False, "act": "silu"},
        # three drafted tokens through both projections, integer weights with zero points
        {"name": "gemv gated int4", "op": "gemv", "M": 3, "N": 2112, "K": 7168, "fmt": "int4", "group": 64, "zeros": True, "gated": True, "act": "silu"},
        # sixteen sequences through the widest projection
        {"name": "gemv wide int4", "op": "gemv", "M": 16, "N": 24576, "K": 7168, "fmt": "int4", "group": 128, "zeros": False, "gated": False, "act": "silu"},
        # the gradients of one small block, both types, a few of them tiny
        {"name": "clip small", "op": "clip", "tensors": 24, "elements": 1 << 18, "types": "both", "sizes": 3, "ratio": 0.37},
        # the gradients of a model: 300 tensors, 400 M elements in both types
        {"name": "clip model", "op": "clip", "tensors": 300, "elements": LARGEST_ELEMENTS, "types": "both", "sizes": 5, "ratio": 0.37},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["gated", "grad", "gemv", "clip"])
    if op == "clip":
        return {"op": op, "tensors": _log_uniform(rng, 1, 300), "elements": _log_uniform(rng, 1000, LARGEST_ELEMENTS),
                "types": rng.choice(["fp32", "bf16", "both"]), "sizes": rng.randrange(1000), "ratio": rng.choice([0.04, 0.37, 2.1])}
    if op == "gemv":
        case = {"op": op, "M": rng.randint(1, 16), "N": _log_uniform(rng, 500, 24576), "K": 128 * rng.randint(4, 56),
                "fmt": rng.choice(["mxfp4", "int4"]), "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                "gated": rng.random() < 0.5, "act": rng.choice(["silu", "gelu"])}
        if case["fmt"] == "mxfp4":
            case["group"], case["zeros"] = 32, False
        return case
    case = {"op": op, "M": _log_uniform(rng, 1, 8192), "N": _log_uniform(rng, 300, 7168), "K": 128 * rng.randint(4, 56),
            "act": rng.choice(["silu", "gelu"])}
    if op == "gated":
        case["out"], case["pow2"] = rng.choice(["bf16", "save", "quant"]), rng.random() < 0.5
        if case["out"] == "quant":
            case["N"] = 128 * max(1, case["N"] // 128)
    case["M"] = max(1, min(case["M"], LARGEST_FLOPS // ((4 if op == "gated" else 8) * case["N"] * case["K"])))
    return case


def _sizes(case):
    """Elements of each gradient: many small ones (norms, biases), few large
    ones (matrices), `elements` in all."""
    r = random.Random(case["sizes"])
    w = [math.exp(r.uniform(0.0, 9.0)) for _ in range(case["tensors"])]
    unit = case["elements"] / sum(w)
    return [max(1, int(x * unit)) for x in w]


def _types(case):
    r = random.Random(case["sizes"] + 1)
    kinds = {"fp32": [torch.float32], "bf16": [torch.bfloat16], "both": [torch.float32, torch.bfloat16]}[case["types"]]
    return [r.choice(kinds) for _ in range(case["tensors"])]


# --------------------------------------------------------------------------
# Inputs.
# --------------------------------------------------------------------------
def _scale(amax, pow2):
    s = amax.clamp_min(1e-4) / 448.0
    return torch.exp2(torch.ceil(torch.log2(s))) if pow2 else s


def _quant_rows(x, pow2):
    """E4M3 codes (M, K) and scales (K/128, M), one per 1x128 group."""
    M, K = x.shape
    s = _scale(x.view(M, K // 128, 128).abs().amax(2), pow2)
    q = (x.view(M, K // 128, 128) / s[..., None]).to(torch.float8_e4m3fn)
    return q.view(M, K).view(torch.uint8), s.t().contiguous()


def _quant_blocks(w, pow2):
    """E4M3 codes (N, K) and scales (ceil(N/128), K/128), one per 128x128 block."""
    N, K = w.shape
    nb = (N + 127) // 128
    full = torch.zeros((nb * 128, K), device=w.device)
    full[:N] = w
    blocks = full.view(nb, 128, K // 128, 128)
    s = _scale(blocks.abs().amax((1, 3)), pow2)
    q = (blocks / s[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * 128, K)[:N]
    return q.contiguous().view(torch.uint8), s.contiguous()


def _weights4(case, g):
    """Packed 4-bit codes (N, K/2), scales and zero points of one weight of
    about 0.02 standard deviation."""
    N, K, G = case["N"], case["K"], case["group"]
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if case["fmt"] == "mxfp4":
        e = torch.randint(118, 122, (K // 128, N, 4), generator=g, device="cuda", dtype=torch.uint8)
        return q, e.view(torch.int32).view(K // 128, N), None
    s = (0.004 * (0.5 + torch.rand((K // G, N), generator=g, device="cuda"))).to(torch.bfloat16)
    z = torch.randint(0, 16, (K // G, N), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    return q, s, z


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    st = {"case": case}
    if case["op"] == "clip":
        # gradients are views of one flat buffer per type, one element apart
        sizes, types = _sizes(case), _types(case)
        for t in (torch.float32, torch.bfloat16):
            total = sum(n + 1 for n, k in zip(sizes, types) if k == t)
            st[str(t)] = normal(total, std=1e-3).to(t)
            st["out " + str(t)] = torch.zeros(total, dtype=t, device="cuda")
        at = {torch.float32: 0, torch.bfloat16: 0}
        st["grads"], st["outs"] = [], []
        for n, t in zip(sizes, types):
            st["grads"].append(st[str(t)][at[t]:at[t] + n])
            st["outs"].append(st["out " + str(t)][at[t]:at[t] + n])
            at[t] += n + 1
        st["max_norm"] = case["ratio"] * 1e-3 * math.sqrt(sum(sizes))     # of the norm, about: below 1 clips
        return st
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gemv":
        st["x"] = normal(M, K).to(torch.bfloat16)
        st["w"] = [_weights4(case, g) for _ in range(2 if case["gated"] else 1)]
        return st
    x = normal(M, K)
    x *= 1.0 + 30.0 * (torch.rand((M, K), generator=g, device="cuda") < 0.001)       # activation outliers
    wg, wu = normal(N, K, std=0.02), normal(N, K, std=0.02)
    if case["op"] == "gated":
        st["x"], st["sa"] = _quant_rows(x, case["pow2"])
        st["wg"], st["sg"] = _quant_blocks(wg, case["pow2"])
        st["wu"], st["su"] = _quant_blocks(wu, case["pow2"])
        return st
    st["x"], st["wg"], st["wu"] = x.to(torch.bfloat16), wg.to(torch.bfloat16), wu.to(torch.bfloat16)
    st["dh"] = normal(M, N, std=1e-2).to(torch.bfloat16)
    st["g"], st["u"] = (normal(M, N, std=0.02 * math.sqrt(K)).to(torch.bfloat16) for _ in range(2))
    return st


# --------------------------------------------------------------------------
# The plain form, in 32 bits.
# --------------------------------------------------------------------------
def _gate(case, g):
    """The activation's value and its derivative's gate: act(g) = g * p."""
    if case["act"] == "silu":
        return 1.0 / (1.0 + torch.exp(-g))
    return 1.0 / (1.0 + torch.exp(-1.5957691216057308 * (g + 0.044715 * g * g * g)))


def _act_grad(case, g):
    p = _gate(case, g)
    if case["act"] == "silu":
        return p * (1.0 + g * (1.0 - p))
    return p + g * p * (1.0 - p) * 1.5957691216057308 * (1.0 + 0.134145 * g * g)


def _rows(q, s):
    return q.view(torch.float8_e4m3fn).float() * s.t().repeat_interleave(128, 1)


def _blocks(q, s):
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)


def _nibbles(q):
    return torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)


def _decode4(case, q, s, z):
    c = _nibbles(q)
    if case["fmt"] == "mxfp4":
        value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)[(c & 7).long()]
        value = torch.where(c >= 8, -value, value)
        e = s.view(torch.uint8).view(s.shape[0], s.shape[1], 4).permute(1, 0, 2).reshape(q.shape[0], -1)
        return value * torch.exp2(e.float() - 127.0).repeat_interleave(32, 1)
    zero = 8.0 if z is None else z.t().float().repeat_interleave(case["group"], 1)
    return (c.float() - zero) * s.t().float().repeat_interleave(case["group"], 1)


def _plain(st):
    case = st["case"]
    if case["op"] == "clip":
        norm = torch.stack([g.float().square().sum() for g in st["grads"]]).sum().sqrt()
        coef = (st["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
        [o.copy_(g.float() * coef) for g, o in zip(st["grads"], st["outs"])]
        return {"norm": norm, "fp32": st["out torch.float32"], "bf16": st["out torch.bfloat16"]}
    if case["op"] == "gemv":
        x = st["x"].float()
        y = x @ _decode4(case, *st["w"][0]).t()
        if case["gated"]:
            y = y * _gate(case, y) * (x @ _decode4(case, *st["w"][1]).t())
        return {"y": y.to(torch.bfloat16)}
    if case["op"] == "gated":
        x = _rows(st["x"], st["sa"])
        g, u = x @ _blocks(st["wg"], st["sg"]).t(), x @ _blocks(st["wu"], st["su"]).t()
        h = g * _gate(case, g) * u
        if case["out"] == "quant":
            q, s = _quant_rows(h, case["pow2"])
            return {"hq": q.view(torch.float8_e4m3fn), "sh": s}
        h16 = h.to(torch.bfloat16)
        return {"h": h16, "g": g.to(torch.bfloat16), "u": u.to(torch.bfloat16)} if case["out"] == "save" else {"h": h16}
    dh, g, u, x = (st[k].float() for k in ("dh", "g", "u", "x"))
    dg, du = dh * u * _act_grad(case, g), dh * g * _gate(case, g)
    return {"dx": (dg @ st["wg"].float() + du @ st["wu"].float()).to(torch.bfloat16),
            "dwg": (dg.t() @ x).to(torch.bfloat16), "dwu": (du.t() @ x).to(torch.bfloat16)}


def run(st):
    """One pass through the case's operator."""
    if not own:
        return _plain(st)
    import fine_grained_block_e4m3_amd as fp8
    case = st["case"]
    if case["op"] == "clip":
        norm = fp8.clip_grad_norm(st["grads"], st["max_norm"], out=st["outs"])
        return {"norm": norm, "fp32": st["out torch.float32"], "bf16": st["out torch.bfloat16"]}
    if case["op"] == "gemv":
        if case["gated"]:
            (wg, sg, zg), (wu, su, zu) = st["w"]
            return {"y": fp8.gated_gemv_w4(st["x"], wg, sg, wu, su, zeros_g=zg, zeros_u=zu, act=case["act"])}
        w, s, z = st["w"][0]
        return {"y": fp8.gemv_w4(st["x"], w, s, zeros=z)}
    if case["op"] == "gated":
        args = [st[k] for k in ("x", "sa", "wg", "sg", "wu", "su")]
        if case["out"] == "quant":
            q, s = fp8.gated_nt_qout(*args, act=case["act"], ue8m0=case["pow2"])
            return {"hq": q.view(torch.float8_e4m3fn), "sh": s}
        if case["out"] == "save":
            h, g, u = fp8.gated_nt(*args, act=case["act"], ue8m0=case["pow2"], save=True)
            return {"h": h, "g": g, "u": u}
        return {"h": fp8.gated_nt(*args, act=case["act"], ue8m0=case["pow2"])}
    dx, dwg, dwu = fp8.gated_nt_grad(*[st[k] for k in ("dh", "g", "u", "x", "wg", "wu")], act=case["act"])
    return {"dx": dx, "dwg": dwg, "dwu": dwu}


def work(case):
    """What one pass cannot do without: inputs read once, outputs written once."""
    if case["op"] == "clip":
        size = {torch.float32: 4, torch.bfloat16: 2}
        n = sum(k * size[t] for k, t in zip(_sizes(case), _types(case)))
        return {"bytes": 2 * n + 4, "flops": 3 * sum(_sizes(case))}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gemv":
        w = N * K // 2 + (K // case["group"]) * N * (1 if case["fmt"] == "mxfp4" else 3 if case["zeros"] else 2)
        both = 2 if case["gated"] else 1
        return {"bytes": both * w + 2 * M * K + 2 * M * N, "flops": both * 2 * M * N * K}
    if case["op"] == "gated":
        read = M * K + 4 * M * (K // 128) + 2 * (N * K + 4 * ((N + 127) // 128) * (K // 128))
        wrote = {"bf16": 2 * M * N, "save": 6 * M * N, "quant": M * N + 4 * M * (N // 128)}[case["out"]]
        return {"bytes": read + wrote, "flops": 4 * M * N * K}
    return {"bytes": 6 * M * N + 4 * M * K + 8 * N * K, "flops": 8 * M * N * K}


# --------------------------------------------------------------------------
# The definitions in 64 bits.
# --------------------------------------------------------------------------
def _e4m3_values():
    """Value of each E4M3 byte: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    b = np.arange(256)
    e, f = (b >> 3) & 15, b & 7
    mag = np.where(e == 0, np.ldexp(f / 8.0, -6), np.ldexp(1.0 + f / 8.0, e - 7))
    return torch.from_numpy(np.where(b >= 128, -mag, mag)).cuda()


def _sigma(case, g):
    t = g if case["act"] == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    return torch.sigmoid(t)


def _exact4(case, q, s, z):
    N, K, G = case["N"], case["K"], case["group"]
    c = torch.empty((N, K), dtype=torch.int64, device="cuda")
    c[:, 0::2], c[:, 1::2] = q & 15, q >> 4
    if case["fmt"] == "mxfp4":
        # two exponent bits (bias 1) and one fraction bit below the sign
        e, f = (c >> 1) & 3, (c & 1).double()
        value = torch.where(e == 0, f / 2, torch.ldexp(1 + f / 2, (e - 1).double())) * (1 - 2 * (c >> 3)).double()
        words = s.long() & 0xFFFFFFFF
        b = torch.stack([(words >> (8 * t)) & 255 for t in range(4)], 1).reshape(K // 32, N).t()
        scale = torch.exp2((b - 127).double())
        return (value.view(N, K // 32, 32) * scale[..., None]).view(N, K)
    zero = torch.full((K // G, N), 8, device="cuda") if z is None else z
    return ((c.view(N, K // G, G).double() - zero.double().t()[..., None]) * s.double().t()[..., None]).view(N, K)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(torch.dot(g.double(), g.double())) for g in st["grads"]))
        coef = min(1.0, st["max_norm"] / (norm + 1e-6))
        outs = {}
        for k, t in (("fp32", torch.float32), ("bf16", torch.bfloat16)):
            keep = torch.zeros_like(st[str(t)], dtype=torch.bool)
            at = 0
            for g in st["grads"]:
                if g.dtype == t:
                    keep[at:at + g.numel()] = True
                    at += g.numel() + 1
            outs[k] = torch.where(keep, st[str(t)].double() * coef, 0.0)
        return {"norm": torch.tensor(norm, dtype=torch.float64), **outs}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gemv":
        x = st["x"].double()
        y = torch.matmul(_exact4(case, *st["w"][0]), x.t()).t()
        if case["gated"]:
            y = y * _sigma(case, y) * torch.matmul(_exact4(case, *st["w"][1]), x.t()).t()
        return {"y": y}
    if case["op"] == "gated":
        lut = _e4m3_values()
        x = (lut[st["x"].long()].view(M, -1, 128) * st["sa"].double().t()[..., None]).view(M, K)

        def weight(q, s):
            rows = torch.arange(N, device="cuda") // 128
            return (lut[q.long()].view(N, -1, 128) * s.double()[rows][..., None]).view(N, K)

        g, u = torch.matmul(x, weight(st["wg"], st["sg"]).t()), torch.matmul(x, weight(st["wu"], st["su"]).t())
        h = g * _sigma(case, g) * u
        if case["out"] == "quant":
            groups = h.view(M, N // 128, 128)
            s = groups.abs().amax(2).clamp_min(1e-4) / 448
            if case["pow2"]:
                s = torch.exp2(torch.ceil(torch.log2(s)))
            return {"hq": (groups / s[..., None]).view(M, N), "sh": s.t()}
        return {"h": h, "g": g, "u": u} if case["out"] == "save" else {"h": h}
    dh, g, u, x, wg, wu = (st[k].double() for k in ("dh", "g", "u", "x", "wg", "wu"))
    g.requires_grad_()
    dact, = torch.autograd.grad((g * _sigma(case, g)).sum(), g)
    g = g.detach()
    dg, du = dh * u * dact, dh * g * _sigma(case, g)
    return {"dx": torch.matmul(dg, wg) + torch.matmul(du, wu), "dwg": torch.matmul(dg.t(), x), "dwu": torch.matmul(du.t(), x)}
