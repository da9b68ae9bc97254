"""Cases, inputs and plain forms of the operators around an adapted MLP block:

norm         RMSNorm of x (+ residual), optionally kept in 8 bits; its backward
keep8        an activation kept in blockwise 8 bits and read back
swiglu8      SwiGLU whose backward reads gate and up from their 8-bit copies
linear_grad8 backward of the adapted NF4 linear layer from its 8-bit input
product4     products of 1 to 16 tokens with a 4-bit weight in any format

``run`` computes the plain form with elementary torch operations in fp32, or,
where the module's ``own`` is true, calls the framework.
"""
from __future__ import annotations

import math
from statistics import NormalDist

import torch

own = False

BLOCK8 = 64                      # values per scale of an 8-bit activation
GROUP = 256                      # block scales per second-level constant
EPS = 1e-5
GAMMA = 2.0                      # LoRA scale alpha / r
TOP8 = {"int8": 127.0, "e4m3": 448.0}
TOP_SCALE = {"e4m3": 448.0, "e5m2": 57344.0, "u8": 255.0}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token in front of a 4096-wide projection: latency
        {"name": "norm_1x4096", "op": "norm", "M": 1, "D": 4096, "res": True, "keep": ""},
        # the MLP workload's 8192 tokens, output kept for the backward
        {"name": "norm_8192x4096_int8", "op": "norm", "M": 8192, "D": 4096, "res": True, "keep": "int8"},
        # the same tokens' backward, with the residual's gradient and the weight's
        {"name": "norm_grad_8192x4096", "op": "norm_grad", "M": 8192, "D": 4096, "res": True},
        # a ragged batch of a small model
        {"name": "norm_grad_513x1088", "op": "norm_grad", "M": 513, "D": 1088, "res": False},
        # an attention projection's 4096-token input, with outlier channels
        {"name": "keep8_4096x4096_e4m3", "op": "keep8", "M": 4096, "D": 4096, "keep": "e4m3"},
        # the MLP workload's hidden activations, forward and backward
        {"name": "swiglu8_8192x11008_int8", "op": "swiglu8", "M": 8192, "D": 11008, "keep": "int8"},
        {"name": "swiglu8_513x1088_e4m3", "op": "swiglu8", "M": 513, "D": 1088, "keep": "e4m3"},
        # the attention projection of the flagship training step
        {"name": "linear_grad8_4096_r16", "op": "linear_grad8", "M": 4096, "N": 4096, "K": 4096, "r": 16,
         "keep": "int8"},
        # decoding one token on a large stored weight with its adapter
        {"name": "product4_nf4_28672x8192_m1", "op": "product4", "M": 1, "N": 28672, "K": 8192, "r": 16,
         "book": "nf4", "block": 64, "scales": "e4m3"},
        # a decoding batch of 16 on groups of 128 with plain scales
        {"name": "product4_int4_8192x28672_m16", "op": "product4", "M": 16, "N": 8192, "K": 28672, "r": 0,
         "book": "int4", "block": 128, "scales": "fp32"},
        # a small weight in the finest groups: latency
        {"name": "product4_fp4_4096x4096_m1", "op": "product4", "M": 1, "N": 4096, "K": 4096, "r": 0,
         "book": "fp4", "block": 16, "scales": "e4m3"},
        # an MLP weight, four sequences, a wide adapter
        {"name": "product4_nf4_11008x4096_m4", "op": "product4", "M": 4, "N": 11008, "K": 4096, "r": 64,
         "book": "nf4", "block": 32, "scales": "u8"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(most, step=64):
        return step * log(1, most // step)

    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "keep8", "swiglu8", "linear_grad8",
                     "product4", "product4", "product4"])
    if op in ("norm", "norm_grad", "keep8", "swiglu8"):
        D = width(16384)
        M = log(1, min(16384, max(1, (8192 * 4096) // D)))
        case = {"op": op, "M": M, "D": D}
        if op == "norm":
            case["keep"] = rng.choice(["", "int8", "e4m3"])
        if op in ("norm", "norm_grad"):
            case["res"] = rng.random() < 0.7
        else:
            case["keep"] = rng.choice(["int8", "e4m3"])
        return case
    if op == "linear_grad8":
        return {"op": op, "M": log(1, 4096), "N": width(4096, 8), "K": width(4096), "r": 8 * rng.randint(1, 16),
                "keep": rng.choice(["int8", "e4m3"])}
    K = width(28672)
    return {"op": op, "M": rng.choice([1, 1, 2, 3, 4, 7, 8, 11, 16]), "N": log(1, min(28672, 28672 * 8192 // K)), "K": K,
            "r": rng.choice([0, 0, 8, 16, 24, 64]), "book": rng.choice(["nf4", "fp4", "int4"]),
            "block": 1 << rng.randint(4, 12), "scales": rng.choice(["fp32", "e4m3", "e5m2", "u8"])}


def work(case):
    op, M = case["op"], case["M"]
    if op in ("norm", "norm_grad", "keep8", "swiglu8"):
        D = case["D"]
        n = M * D
        if op == "norm":        # x (and r) in, y (and h, and the values kept) out
            return {"bytes": n * (4 + (4 if case["res"] else 0) + (2 if case["keep"] else 0)) + 4 * D, "flops": 6 * n}
        if op == "norm_grad":   # dy, h (and dr) in, dx out, the weight and its gradient
            return {"bytes": n * (6 + (2 if case["res"] else 0)) + 8 * D, "flops": 12 * n}
        if op == "keep8":       # x in, the values kept and their scales out
            return {"bytes": n * 4 + n // BLOCK8 * 4, "flops": 4 * n}
        return {"bytes": n * 12, "flops": 30 * n}   # g, u, dh in, h, dg, du out
    N, K, r = case["N"], case["K"], case["r"]
    if op == "linear_grad8":
        stored = N * K / 2 + N * K / 64 + N * K / 64 / GROUP * 4
        x8 = M * K + M * K / BLOCK8 * 4
        return {"bytes": 2 * M * N + x8 + stored + 2 * M * K + 4 * r * (N + K) + 4 * M * r,
                "flops": 2 * M * N * K + 4 * M * r * (N + K)}
    blocks = -(-N * K // case["block"])
    scale = blocks * 4 if case["scales"] == "fp32" else blocks + blocks / GROUP * 4
    return {"bytes": N * K / 2 + scale + 2 * M * (N + K) + 2 * r * (N + K),
            "flops": 2 * M * N * K + 2 * M * r * (N + K)}


# ------------------------------------------------------------------ inputs
def codebook(name):
    """Ascending codes in [-1, 1], each an fp32 value."""
    if name == "nf4":
        q = NormalDist().inv_cdf
        d = 0.5 * ((1 - 1 / 30) + (1 - 1 / 32))
        v = [-q(d - j * (d - 0.5) / 7) for j in range(7)] + [0.0] + [q(d - j * (d - 0.5) / 8) for j in range(8)]
        v = [x / q(d) for x in v]
    elif name == "fp4":
        m = [0.5, 1, 1.5, 2, 3, 4, 6]
        v = [-x / 6 for x in m] + [0.0] + [x / 6 for x in m]
    else:
        v = [k / 7 for k in range(-7, 8)]
    return torch.tensor(sorted(v), dtype=torch.float32).tolist()


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activation(gen, M, D):
    """bf16 tokens with a few outlier channels, and padding rows of zeros."""
    x = _normal(gen, M, D)
    x[:, :: 101] *= 12.0
    if M > 8:
        x[M - M // 16:] = 0.0
    return x.to(torch.bfloat16)


def _store8(x, keep):
    """The 8-bit copy of a bf16 activation: codes and fp32 scales."""
    b = x.float().reshape(-1, BLOCK8)
    c = b.abs().amax(1, keepdim=True)
    q = b * TOP8[keep] / torch.where(c > 0, c, 1.0)
    codes = torch.round(q).to(torch.int8) if keep == "int8" else q.to(torch.float8_e4m3fn)
    return codes.reshape(-1), (c / TOP8[keep]).reshape(-1)


def _store4(w, book, block, scales):
    """Packed indices, block scales and second-level constants of a weight."""
    codes = torch.tensor(codebook(book), device=w.device)
    mids = ((codes[1:].double() + codes[:-1].double()) / 2).float()
    n = w.numel()
    pad = (-n) % block
    b = torch.nn.functional.pad(w.reshape(-1), (0, pad)).reshape(-1, block)
    c = b.abs().amax(1)
    idx = torch.bucketize(b / torch.where(c > 0, c, 1.0)[:, None], mids, out_int32=True).to(torch.uint8).reshape(-1, 2)
    packed = idx[:, 0] | (idx[:, 1] << 4)
    if scales == "fp32":
        return packed, c, None
    g = torch.nn.functional.pad(c, (0, (-c.numel()) % GROUP)).reshape(-1, GROUP)
    meta = g.amax(1) / TOP_SCALE[scales]
    x = (g / torch.where(meta > 0, meta, 1.0)[:, None]).reshape(-1)[: c.numel()]
    if scales == "u8":
        code = torch.round(x).clamp(max=255).to(torch.uint8)
    else:
        t = torch.float8_e4m3fn if scales == "e4m3" else torch.float8_e5m2
        code = x.clamp(max=TOP_SCALE[scales]).to(t).view(torch.uint8)
    return packed, code, meta


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M = case["op"], case["M"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        D = case["D"]
        s["x"] = _activation(gen, M, D)
        s["res"] = _activation(gen, M, D) if case["res"] else None
        s["w"] = 1.0 + 0.2 * _normal(gen, D)
        if op == "norm_grad":
            s["dy"] = _normal(gen, M, D).to(torch.bfloat16)
    elif op == "keep8":
        s["x"] = _activation(gen, M, case["D"])
    elif op == "swiglu8":
        D = case["D"]
        s["g"], s["u"] = (_activation(gen, M, D) for _ in range(2))
        s["dh"] = _normal(gen, M, D).to(torch.bfloat16)
    elif op == "linear_grad8":
        N, K, r = case["N"], case["K"], case["r"]
        x = _activation(gen, M, K)
        s["codes"], s["xs"] = _store8(x, case["keep"])
        s["dy"] = _normal(gen, M, N).to(torch.bfloat16)
        s["w"] = _store4(0.02 * _normal(gen, N, K), "nf4", 64, "e4m3")
        s["A"] = (_normal(gen, r, K) / math.sqrt(K)).to(torch.bfloat16)
        s["B"] = (0.01 * _normal(gen, N, r)).to(torch.bfloat16)
        s["T"] = x.float() @ s["A"].float().t()
    else:
        N, K, r = case["N"], case["K"], case["r"]
        s["x"] = _activation(gen, M, K)
        s["w"] = _store4(0.015 * _normal(gen, N, K), case["book"], case["block"], case["scales"])
        s["A"] = (_normal(gen, r, K) / math.sqrt(K)).to(torch.bfloat16) if r else None
        s["B"] = (0.01 * _normal(gen, N, r)).to(torch.bfloat16) if r else None
    return s


# -------------------------------------------------------------- plain form
def _load8(codes, scales, shape, t=torch.float32):
    return (codes.to(t).reshape(-1, BLOCK8) * scales.to(t)[:, None]).reshape(shape)


def _load4(w, N, K, book, block, scales, t=torch.float32):
    packed, sc, meta = w
    codes = torch.tensor(codebook(book), device=packed.device, dtype=t)
    q = codes[torch.stack((packed & 15, packed >> 4), 1).reshape(-1).long()]
    if scales == "fp32":
        c = sc.to(t)
    else:
        v = sc if scales == "u8" else sc.view(torch.float8_e4m3fn if scales == "e4m3" else torch.float8_e5m2)
        c = v.to(t) * meta.to(t).repeat_interleave(GROUP)[: sc.numel()]
    return (q.reshape(-1, block) * c[:, None]).reshape(-1)[: N * K].reshape(N, K)


def _plain(s):
    case = s["case"]
    op, M, bf = case["op"], case["M"], torch.bfloat16
    if op == "norm":
        h = (s["x"].float() + s["res"].float()).to(bf) if case["res"] else s["x"]
        f = h.float()
        y = (f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * s["w"]).to(bf)
        out = {"y": y, "h": h} if case["res"] else {"y": y}
        if case["keep"]:
            out["y8"] = _load8(*_store8(y, case["keep"]), y.shape).to(bf)
        return out
    if op == "norm_grad":
        h, dy = s["x"].float(), s["dy"].float()
        rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        wd = dy * s["w"]
        dx = rstd * (wd - h * rstd.square() * (wd * h).mean(1, keepdim=True))
        if case["res"]:
            dx = dx + s["res"].float()
        return {"dx": dx.to(bf), "dw": (dy.double() * h * rstd).sum(0).float()}
    if op == "keep8":
        codes, scales = _store8(s["x"], case["keep"])
        return {"x": _load8(codes, scales, s["x"].shape).to(bf), "scales": scales}
    if op == "swiglu8":
        h = (s["g"].float() * torch.sigmoid(s["g"].float()) * s["u"].float()).to(bf)
        g = _load8(*_store8(s["g"], case["keep"]), h.shape).to(bf).float()
        u = _load8(*_store8(s["u"], case["keep"]), h.shape).to(bf).float()
        sg, dh = torch.sigmoid(g), s["dh"].float()
        return {"h": h, "dg": (dh * u * (sg * (1 + g * (1 - sg)))).to(bf), "du": (dh * g * sg).to(bf)}
    N, K, r = case["N"], case["K"], case["r"]
    if op == "linear_grad8":
        # the adapter's gradients go to bf16, the precision its products are made in
        x = _load8(s["codes"], s["xs"], (M, K)).to(bf).float()
        w = _load4(s["w"], N, K, "nf4", 64, "e4m3").to(bf).float()
        dy, A, B = s["dy"].float(), s["A"].float(), s["B"].float()
        u = dy @ B
        return {"dx": (dy @ w + GAMMA * u @ A).to(bf), "dA": (GAMMA * u.t() @ x).to(bf),
                "dB": (GAMMA * dy.t() @ s["T"]).to(bf)}
    x = s["x"].float()
    y = x @ _load4(s["w"], N, K, case["book"], case["block"], case["scales"]).t()
    if r:
        y = y + GAMMA * (x @ s["A"].float().t()) @ s["B"].float().t()
    return y.to(bf)


# ------------------------------------------------------- the framework's calls
_scale_names = {"fp32": "QLORA_SCALES_FP32", "e4m3": "QLORA_SCALES_E4M3", "e5m2": "QLORA_SCALES_E5M2",
                "u8": "QLORA_SCALES_U8"}


def _framework(s):
    import bit_nf4_quantised_b200 as q

    case = s["case"]
    op, M, bf = case["op"], case["M"], torch.bfloat16
    code = {"int8": q.QLORA_ACT8_INT8, "e4m3": q.QLORA_ACT8_E4M3}.get(case.get("keep"))
    if op == "norm":
        q8 = q.empty_act8(M, case["D"], code) if case["keep"] else None
        y, h = q.qlora_rmsnorm_forward(s["x"], s["w"], EPS, residual=s["res"], q8=q8)
        out = {"y": y, "h": h} if case["res"] else {"y": y}
        if case["keep"]:
            out["y8"] = q.qlora_act8_dequantize(q8)
        return out
    if op == "norm_grad":
        dx, dw = q.qlora_rmsnorm_backward(s["dy"], s["x"], s["w"], EPS, dres=s["res"])
        return {"dx": dx, "dw": dw}
    if op == "keep8":
        x8 = q.qlora_act8_quantize(s["x"], code)
        return {"x": q.qlora_act8_dequantize(x8), "scales": x8.scales}
    if op == "swiglu8":
        h, g8, u8 = q.qlora_swiglu_forward_act8(s["g"], s["u"], code)
        dg, du = q.qlora_swiglu_backward_act8(s["dh"], g8, u8)
        return {"h": h, "dg": dg, "du": du}
    N, K, r = case["N"], case["K"], case["r"]
    if op == "linear_grad8":
        x8 = q.Act8(s["codes"], s["xs"], M, K, code)
        w = q.NF4Tensor(*s["w"], N, K)
        dx, dA, dB = q.qlora_linear_backward_act8(s["dy"], x8, w, s["A"], s["B"], GAMMA, T_saved=s["T"])
        return {"dx": dx, "dA": dA.to(bf), "dB": dB.to(bf)}
    if "fmt" not in s:      # a serving program keeps its weight's format
        s["fmt"] = q.Format(tuple(codebook(case["book"])), case["block"], getattr(q, _scale_names[case["scales"]]))
    return q.qlora_linear_fmt_forward(s["x"], *s["w"], N, s["fmt"], A=s["A"], B=s["B"], scale=GAMMA)


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, M, d = case["op"], case["M"], torch.float64

    def kept(x):
        b = x.to(d).reshape(-1, BLOCK8)
        c = b.abs().max(1, keepdim=True).values
        top = TOP8[case["keep"]]
        q = torch.nan_to_num(b / c * top if case["keep"] == "e4m3" else torch.round(b * top / c), nan=0.0)
        q = q.to(torch.float8_e4m3fn).to(d) if case["keep"] == "e4m3" else q
        return (q * c / top).reshape(x.shape), (c / top).reshape(-1)

    if op == "norm":
        h = s["x"].to(d)
        if case["res"]:
            h = (h + s["res"].to(d)).to(torch.bfloat16).to(d)      # the residual stream is bf16
        y = h * s["w"].to(d) / torch.sqrt((h * h).sum(1, keepdim=True) / case["D"] + EPS)
        out = {"y": y, "h": h} if case["res"] else {"y": y}
        if case["keep"]:
            out["y8"] = kept(y.to(torch.bfloat16))[0]
        return out
    if op == "norm_grad":
        h, dy, w = s["x"].to(d), s["dy"].to(d), s["w"].to(d)
        ms = (h * h).sum(1, keepdim=True) / case["D"] + EPS
        n = h / torch.sqrt(ms)
        t = dy * w
        dx = (t - n * (t * n).sum(1, keepdim=True) / case["D"]) / torch.sqrt(ms)
        return {"dx": dx + s["res"].to(d) if case["res"] else dx, "dw": torch.einsum("md,md->d", dy, n)}
    if op == "keep8":
        x, scales = kept(s["x"])
        return {"x": x, "scales": scales}
    if op == "swiglu8":
        def silu(z):
            return z / (1 + torch.exp(-z))
        (g, _), (u, _), dh = kept(s["g"]), kept(s["u"]), s["dh"].to(d)
        sg = 1 / (1 + torch.exp(-g))
        return {"h": silu(s["g"].to(d)) * s["u"].to(d), "dg": dh * u * (sg + silu(g) * (1 - sg)), "du": dh * silu(g)}
    N, K, r = case["N"], case["K"], case["r"]
    if op == "linear_grad8":
        w = _load4(s["w"], N, K, "nf4", 64, "e4m3", d).to(torch.bfloat16).to(d)     # W~ is bf16 by its definition
        dy, A, B = s["dy"].to(d), s["A"].to(d), s["B"].to(d)
        x = _load8(s["codes"], s["xs"], (M, K), d)
        return {"dx": torch.mm(dy, w) + GAMMA * torch.mm(torch.mm(dy, B), A),
                "dA": GAMMA * torch.mm(torch.mm(B.t(), dy.t()), x), "dB": GAMMA * torch.mm(dy.t(), s["T"].to(d))}
    x = s["x"].to(d)
    y = torch.mm(x, _load4(s["w"], N, K, case["book"], case["block"], case["scales"], d).t())
    return y if not r else y + GAMMA * torch.mm(torch.mm(x, s["A"].to(d).t()), s["B"].to(d).t())
